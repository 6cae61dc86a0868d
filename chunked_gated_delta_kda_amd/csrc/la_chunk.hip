// la_chunk.hip -- chunked linear attention with a decay for each head (gfx950).
//
// With a = exp(log_decay[h]) and the state S [D1, D2] of a (sequence, head),
// one pass computes, token after token,
//   S <- a S + y_t z_t^T,   O_t = S^T x_t
// (in reverse, with late = 1, S^T x_t comes before the decay and the token's
// own decay after it).  Over a chunk of C = 64 positions:
//   O_i = x_scale a^(i+1-late) S^T x_i + in_scale sum_{j<=i} a^(i-j) (x_i . y_j) z_j
//   S  <- a^n S + z_scale sum_j a^(n-1-j+late) y_j z_j^T.
// The forward pass is (x, y, z) = (q, k, v).  With E_t the gradient of S_t
// from later tokens and R_t = E_t + scale q_t do_t^T,
//   dq_t = scale S_t do_t   the forward pass (do, v, k) on S^T,
//   dv_t = R_t^T k_t        the reversed pass (k, q, do) on R,
//   dk_t = R_t v_t          the reversed pass (v, do, q) on R^T,
//   E_(t-1) = a R_t         (the reversed passes' state; E_(-1) = dh0),
// so one kernel serves all four.
//
// One workgroup of eight waves per (segment, head), alone on its CU (160 KB of LDS):
//  - four waves move rows: every chunk, x and y two chunks ahead and z one ahead from
//    memory into LDS (loaded two chunks before that), the outputs from LDS to memory,
//    whole rows at a time; and they form P^T = in_scale a^(i-j) (x_i . y_j) of the
//    next chunk (16x16x32 MFMAs on the raw bf16 rows), left in LDS as operands;
//  - four waves keep the state, D2 / 4 columns each, in fp32 accumulators.  Rounded,
//    they are the operand of S^T x as they are, so the state never leaves its wave;
//    y and z are read by transposing reads as operands that contract over tokens.
// One barrier a chunk.
//
// What bounds it: with every CU busy, HBM: 16 sequences of 256 to 8192 tokens, 32 heads
// of 128 x 128, take 591 to 612 us for 2.55 GB, 4.2 to 4.3 TB/s, where a copy of 2 GiB
// reaches 4.9.  With 64
// workgroups the issue of instructions: a chunk costs a SIMD 152 products of 16 cycles
// and about 700 other vector instructions, which overlap for a fifth only, 2.6 us in
// all.  Measured on the way there (the packed batch):
// 32 columns a workgroup, z in 64-byte pieces, 820 us; eight state waves of 16 columns,
// which read x and y from LDS twice as often, 615; products and conversions in the
// compiler's own order 616.
//
// Precision: raw bf16 operands; P and the copy of S are rounded to bf16 once each
// (outputs are bf16).  The state itself is fp32 to its last bits where it is returned:
// a token's decayed z is split into three bf16 terms (24 bits), so every product of
// the update is exact, and the decays of the chunks do not drift from a's powers
// (ChunkDecay).  Where no state is returned two terms (16 bits) are enough, since
// the state is then only read through its rounding to 8 bits (gradients of 24 packed
// sequences, 16 heads of 128 x 64: 166 -> 158 us).
#include "la_device.h"

namespace kda {

// LDS of a workgroup: three tiles each of x, y, z and two sets of P
template <int D1, int D2, bool STATES>
constexpr int lds_bytes() {
    return 3 * LC * (STATES ? D1 + D2 : 2 * D1 + D2) * 2 + (STATES ? 0 : 2 * 6 * 64 * 16);
}

template <int D1, int D2, int TERMS, bool STATES>
__device__ __forceinline__ void chunk_pass(const LaArgs& a, const LaPass& p, int slot, int h, unsigned char* lds) {
    constexpr int NC = D2 / 64;            // 16-column tiles of each of the four state waves
    constexpr int KS = D1 / 32;            // 16x16x32 steps over D1
    constexpr int NT = D1 / 16;            // state tiles of a wave
    // the four waves that move rows: 16-byte pieces of an x or y tile (of a z tile)
    // per thread, threads per row, rows that they cover at once
    constexpr int RV = D1 / 32, RT = D1 / 8, RROWS = 256 / RT;
    constexpr int ZV = D2 / 32, ZT = D2 / 8, ZROWS = 256 / ZT;
    constexpr int PT = 3;                  // tiles of P per wave, at most
    bf16(*const ytile)[LC * D1] = reinterpret_cast<bf16(*)[LC * D1]>(lds);
    bf16(*const ztile)[LC * D2] = reinterpret_cast<bf16(*)[LC * D2]>(ytile + 3);
    bf16(*const xtile)[LC * D1] = reinterpret_cast<bf16(*)[LC * D1]>(ztile + 3);
    bf16x8(*const pfrag)[6][64] = reinterpret_cast<bf16x8(*)[6][64]>(xtile + 3);

    const int H = a.s.H;
    Seg sg;
    if (!find_seg(a.s, slot, sg)) return;
    const float ld = head_log_decay(a.log_decay, h);
    const float l2 = ld * LOG2E;
    if constexpr (STATES) {
        if (sg.p1 == sg.len) return;  // nobody enters from a sequence's last segment
    }

    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool mover = wave < 4;
    const int late = p.reverse ? 1 : 0;

    if (!STATES && a.s.cu && sg.p0 == 0 && (sg.n == 0 || sg.n == a.s.n_seqs - 1)) {
        // rows outside every sequence: zeros
        auto zero_rows = [&](int lo, int hi) {
            for (int t = lo + (int)threadIdx.x / ZT; t < hi; t += 512 / ZT)
                *reinterpret_cast<u32x4*>(p.o + ((int64_t)t * H + h) * D2 + 8 * (threadIdx.x % ZT)) = u32x4{0, 0, 0, 0};
        };
        if (sg.n == 0) zero_rows(0, sg.t0);
        if (sg.n == a.s.n_seqs - 1) zero_rows(sg.t0 + sg.len, a.s.T);
    }

    // ---- rows of x, y, z of a chunk: a uniform base and a 32-bit byte offset
    // per row.  Positions behind the segment's end read its last row, whose
    // weight in the state is then zero and whose output is not stored, and
    // chunks behind the last one read that one: every load is unconditional.
    // (In reverse the base is the chunk's last position, the lowest address.)
    const int np = sg.p1 - sg.p0, nc = (np + LC - 1) / LC;
    const int64_t first = p.reverse ? (int64_t)sg.t0 + sg.len - LC - sg.p0 : (int64_t)sg.t0 + sg.p0;
    const int64_t x_first = (first * H + h) * (D1 * 2), z_first = (first * H + h) * (D2 * 2);
    const int64_t x_step = (p.reverse ? -1 : 1) * (int64_t)LC * H * (D1 * 2);
    const int64_t z_step = (p.reverse ? -1 : 1) * (int64_t)LC * H * (D2 * 2);
    const uint32_t x_row = (uint32_t)H * (D1 * 2), z_row = (uint32_t)H * (D2 * 2);
    auto offset = [&](int row, uint32_t bytes) { return (uint32_t)(p.reverse ? LC - 1 - row : row) * bytes; };
    auto load16 = [](const char* base, uint32_t o) { return *reinterpret_cast<const u32x4*>(base + o); };
    const char* const x_ptr = reinterpret_cast<const char*>(p.x) + x_first;
    const char* const y_ptr = reinterpret_cast<const char*>(p.y) + x_first;
    const char* const z_ptr = reinterpret_cast<const char*>(p.z) + z_first;
    char* const o_ptr = reinterpret_cast<char*>(p.o) + z_first;

    // LDS reads of a tile's rows 16 t + r, channels 32 j + 8 g (an operand that
    // contracts over channels)
    int row_off[KS];
#pragma unroll
    for (int j = 0; j < KS; ++j) row_off[j] = r * D1 + 8 * ((4 * j + g) ^ swizzle<D1>(r));
    auto row_frag = [&](const bf16* tile, int t, int j) __attribute__((always_inline)) {
        return *reinterpret_cast<const bf16x8*>(tile + 16 * t * D1 + row_off[j]);
    };

    if (mover) {
        if (nc == 0) return;
        // ================= rows and P.  In interval c these waves leave x and y of
        // chunk c + 2, z of c + 1 and P of c + 1 in LDS, and store the outputs of
        // chunk c - 1, which the state waves left in place of its z.
        const int tid = threadIdx.x;
        const int r_row = tid / RT, r_unit = tid % RT, z_trow = tid / ZT, z_unit = tid % ZT;
        auto load_rows = [&](const char* ptr, int c, u32x4 (&v)[RV]) __attribute__((always_inline)) {
            c = min(c, nc - 1);
            const int last = np - 1 - c * LC;
            uint32_t o[RV];
#pragma unroll
            for (int i = 0; i < RV; ++i) o[i] = offset(r_row + i * RROWS, x_row);
            if (last < LC - 1) {
#pragma unroll
                for (int i = 0; i < RV; ++i) o[i] = offset(min(r_row + i * RROWS, last), x_row);
            }
#pragma unroll
            for (int i = 0; i < RV; ++i) v[i] = load16(ptr + c * x_step, o[i] + 16 * r_unit);
        };
        auto load_z = [&](int c, u32x4 (&v)[ZV]) __attribute__((always_inline)) {
            c = min(c, nc - 1);
            const int last = np - 1 - c * LC;
            uint32_t o[ZV];
#pragma unroll
            for (int i = 0; i < ZV; ++i) o[i] = offset(z_trow + i * ZROWS, z_row);
            if (last < LC - 1) {
#pragma unroll
                for (int i = 0; i < ZV; ++i) o[i] = offset(min(z_trow + i * ZROWS, last), z_row);
            }
#pragma unroll
            for (int i = 0; i < ZV; ++i) v[i] = load16(z_ptr + c * z_step, o[i] + 16 * z_unit);
        };
        auto put_rows = [&](bf16* tile, const u32x4 (&v)[RV]) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < RV; ++i) {
                const int row = r_row + i * RROWS;
                *reinterpret_cast<u32x4*>(tile + row * D1 + 8 * (r_unit ^ swizzle<D1>(row))) = v[i];
            }
        };
        auto z_piece = [&](int c, int i) __attribute__((always_inline)) {
            const int row = z_trow + i * ZROWS;
            return reinterpret_cast<u32x4*>(&ztile[c % 3][row * D2 + 8 * (z_unit ^ swizzle<D2>(row))]);
        };
        auto put_z = [&](int c, const u32x4 (&v)[ZV]) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < ZV; ++i) *z_piece(c, i) = v[i];
        };
        auto store_rows = [&](int c, auto full) __attribute__((always_inline)) {
            u32x4 v[ZV];
#pragma unroll
            for (int i = 0; i < ZV; ++i) v[i] = *z_piece(c, i);
#pragma unroll
            for (int i = 0; i < ZV; ++i) {
                const int row = z_trow + i * ZROWS;
                if (decltype(full)::value || c * LC + row < np)
                    *reinterpret_cast<u32x4*>(o_ptr + c * z_step + (offset(row, z_row) + 16 * z_unit)) = v[i];
            }
        };
        // P^T of chunk c, by tiles (key tile k, query tile q), left as halves of the
        // operands of P z: (q, key tiles 0 and 1), and for q = 2, 3 (q, key tiles 2 and 3)
        int pk[PT], pq[PT];
        float dec[PT][4];
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            const int t = wave + 4 * i;  // 0..3: the first row of keys, then 4..6, 7..8, 9
            pk[i] = t < 4 ? 0 : t < 7 ? 1 : t < 9 ? 2 : 3;
            pq[i] = t < 4 ? t : t < 7 ? t - 3 : t < 9 ? t - 5 : 3;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                dec[i][e] = exp2_hw(max(16 * (pq[i] - pk[i]) + r - 4 * g - e, 0) * l2) * p.in_scale;
        }
        auto scores = [&](int c) __attribute__((always_inline)) {
            const bf16* xt = xtile[c % 3];
            const bf16* yt = ytile[c % 3];
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                if (i == 2 && wave >= 2) continue;
                floatx4 t;
#pragma unroll
                for (int j = 0; j < KS; ++j)
                    t = mfma32(row_frag(yt, pk[i], j), row_frag(xt, pq[i], j), j ? t : floatx4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    t[e] *= dec[i][e];
                    if (pk[i] == pq[i] && r < 4 * g + e) t[e] = 0.f;
                }
                const int f = pk[i] < 2 ? pq[i] : pq[i] + 2;
                reinterpret_cast<bf16x4*>(&pfrag[c & 1][f][lane])[pk[i] & 1] = to_bf16x4(t);
            }
        };

        u32x4 xr[2][RV], yr[2][RV], zr[2][ZV];  // two chunks ahead
        {
            u32x4 x0[RV], y0[RV], z0[ZV], x1[RV], y1[RV];
            if constexpr (!STATES) load_rows(x_ptr, 0, x0);
            load_rows(y_ptr, 0, y0);
            load_z(0, z0);
            if constexpr (!STATES) load_rows(x_ptr, 1, x1);
            load_rows(y_ptr, 1, y1);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                load_z(1 + k, zr[k]);
                if constexpr (!STATES) load_rows(x_ptr, 2 + k, xr[k]);
                load_rows(y_ptr, 2 + k, yr[k]);
            }
            if constexpr (!STATES) put_rows(xtile[0], x0);
            put_rows(ytile[0], y0);
            put_z(0, z0);
            if constexpr (!STATES) put_rows(xtile[1], x1);
            put_rows(ytile[1], y1);
            // the halves that no tile of P fills
            if (!STATES && wave < 2) {
                reinterpret_cast<bf16x4*>(&pfrag[wave][0][lane])[1] = bf16x4{};
                reinterpret_cast<bf16x4*>(&pfrag[wave][4][lane])[1] = bf16x4{};
            }
        }
        __syncthreads();
        if constexpr (!STATES) {
            scores(0);
            __syncthreads();
        }
        auto interval = [&](int c, u32x4 (&x)[RV], u32x4 (&y)[RV], u32x4 (&z)[ZV]) __attribute__((always_inline)) {
            if constexpr (!STATES) {
                if (c > 0) store_rows(c - 1, std::true_type{});
                scores(c + 1);
                put_rows(xtile[(c + 2) % 3], x);
            }
            put_rows(ytile[(c + 2) % 3], y);
            put_z(c + 1, z);
            if constexpr (!STATES) load_rows(x_ptr, c + 4, x);
            load_rows(y_ptr, c + 4, y);
            load_z(c + 3, z);
            __syncthreads();
        };
        int c = 0;
        for (; c + 2 < nc; c += 2) {
            interval(c, xr[0], yr[0], zr[0]);
            interval(c + 1, xr[1], yr[1], zr[1]);
        }
        if (c + 1 < nc) interval(c, xr[0], yr[0], zr[0]);
        if (!STATES && nc > 1) store_rows(nc - 2, std::true_type{});
        __syncthreads();
        if constexpr (!STATES) store_rows(nc - 1, std::false_type{});
        return;
    }

    // ================= the state.  Wave w owns columns 16 NC w .. over all rows:
    // accumulator element i of tile (n, kt) is row channel(kt, 4 g + i), column
    // 16 (NC w + n) + r; so S, rounded, is the operand of S^T x without leaving its wave.
    const int w = wave - 4;
    floatx4 S[NC][NT];
    const int64_t state_at = (int64_t)(16 * NC * w + r) * p.col;
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int kt = 0; kt < NT; ++kt) S[n][kt] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (!STATES && p.s_in) {
        const float* t = p.s_in + ((int64_t)(p.s_in_slots ? slot : sg.n) * H + h) * (D1 * D2) + state_at;
        auto load = [&](int row) __attribute__((always_inline)) {
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int kt = 0; kt < NT; ++kt) S[n][kt] = load_state(t + 16 * n * p.col, tile_channel(kt, 4 * g), row);
        };
        if (p.row == 1) load(1);
        else load(p.row);
    }
    if (nc > 0) {
        ChunkDecay chunk_decay(ld);
        float decay, wt[2][8];
        // (a chunk's decay and its tokens' weights)
        auto set_chunk = [&](int n) __attribute__((always_inline)) {
            if (n < LC) decay = exp2_hw(n * l2);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int t = 32 * m + 16 * (e >> 2) + 4 * g + (e & 3);
                    wt[m][e] = t < n ? exp2_hw((n - 1 - t + late) * l2) * p.z_scale : 0.f;
                }
        };
        set_chunk(LC);
        float up[4];  // decay of the entering state at query 16 q + r
#pragma unroll
        for (int q = 0; q < 4; ++q) up[q] = exp2_hw((16 * q + r + 1 - late) * l2) * p.x_scale;
        // transposing reads of y (tiles 2 T and 2 T + 1) and of the wave's z columns
        const int t_row = 4 * g + (r >> 2);
        int y_off[NT / 2], z_off[NC], o_off[NC];
#pragma unroll
        for (int T = 0; T < NT / 2; ++T) y_off[T] = t_row * D1 + 8 * ((4 * T + (r & 3)) ^ swizzle<D1>(t_row));
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            z_off[n] = t_row * D2 + 8 * ((2 * (NC * w + n) + ((r & 3) >> 1)) ^ swizzle<D2>(t_row)) + 4 * (r & 1);
            o_off[n] = r * D2 + 8 * ((2 * (NC * w + n) + (g >> 1)) ^ swizzle<D2>(r)) + 4 * (g & 1);
        }

        __syncthreads();
        if constexpr (!STATES) __syncthreads();
        // S, rounded: the operands of S^T x
        bf16x8 sf[NC][KS];
        auto round_state = [&](int n, int j) __attribute__((always_inline)) {
            if constexpr (!STATES) {
                sf[n][j] = join(to_bf16x4(S[n][2 * j]), to_bf16x4(S[n][2 * j + 1]));
                pin(sf[n][j]);
            }
        };
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int j = 0; j < KS; ++j) round_state(n, j);
        auto decay_tile = [&](int n, int kt) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) S[n][kt][i] *= decay;
            pin(S[n][kt]);
        };

        // One chunk.  A wave is alone with one mover on its SIMD, so the order of its
        // instructions has to keep the matrix pipe busy: a product issues in a quarter
        // of the cycles that it takes, and each is followed by the few conversions
        // that fill the rest (FENCE keeps the compiler from gathering them); operands
        // are read from LDS a step ahead.
        for (int c = 0; c < nc; ++c) {
            bf16* zt = ztile[c % 3];
            const bf16* yt = ytile[c % 3];
            bf16x8 zf[NC][2], yf[3];
            floatx4 acc[NC][4];
            u32x4 term[2][NC][TERMS];
            decay = chunk_decay.step();
            if (c == nc - 1 && np - c * LC < LC) set_chunk(np - c * LC);
            auto read_y = [&](int i) __attribute__((always_inline)) {
                const bf16* y0 = yt + 32 * (i / NT) * D1 + y_off[i % NT / 2] + 4 * (i & 1);
                yf[i % 3] = join(read_t(y0), read_t(y0 + 16 * D1));
            };
            // z of half a chunk, decayed to the chunk's end, as bf16 terms, in 16 NC steps
            float v0, v1;
            auto split = [&](int m, int step) __attribute__((always_inline)) {
                const int n = step / 16, e = step / 4 % 4, q = step % 4;
                if (q == 0) {
                    const uint32_t raw = __builtin_bit_cast(u32x4, zf[n][m])[e];
                    v0 = decayed(bf_lo(raw), wt[m][2 * e]);
                    v1 = decayed(bf_hi(raw), wt[m][2 * e + 1]);
                } else if (q <= TERMS) {
                    uint32_t two = take_term(v0, v1);
                    pin(two);
                    term[m][n][q - 1][e] = two;
                }
            };
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NC; ++n)
                    zf[n][m] = join(read_t(zt + z_off[n] + 32 * m * D2), read_t(zt + z_off[n] + (32 * m + 16) * D2));
            // S^T x (D rows are the wave's columns, D columns the queries), and the first split
            if constexpr (!STATES) {
                const bf16* xt = xtile[c % 3];
                bf16x8 xf[2][4], pf[6];
#pragma unroll
                for (int q = 0; q < 4; ++q) xf[0][q] = row_frag(xt, q, 0);
                FENCE;
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    if (j + 1 < KS) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) xf[(j + 1) & 1][q] = row_frag(xt, q, j + 1);
                    } else {
#pragma unroll
                        for (int q = 0; q < 6; ++q) pf[q] = pfrag[c & 1][q][lane];
                    }
#pragma unroll
                    for (int i = 0; i < 4 * NC; ++i) {
                        const int q = i / NC, n = i % NC, k = j * 4 * NC + i;
                        acc[n][q] = mfma32(sf[n][j], xf[j & 1][q], j ? acc[n][q] : floatx4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                        for (int u = 0; u < 4 / KS; ++u) split(0, 4 / KS * k + u);
                        FENCE;
                    }
                }
                // P z, and the state's decay
                read_y(0);
                read_y(1);
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int n = 0; n < NC; ++n) acc[n][q] *= up[q];
                FENCE;
#pragma unroll
                for (int i = 0; i < 6 * NC; ++i) {
                    const int q = i / NC < 4 ? i / NC : i / NC - 2, n = i % NC;
                    acc[n][q] = mfma32(zf[n][i / NC < 4 ? 0 : 1], pf[i / NC], acc[n][q]);
#pragma unroll
                    for (int t = 0; t < NC * NT; ++t)
                        if (t * 6 / NT == i) decay_tile(t % NC, t / NC);
                    FENCE;
                }
            } else {
                read_y(0);
                read_y(1);
#pragma unroll
                for (int k = 0; k < 16 * NC; ++k) split(0, k);
#pragma unroll
                for (int t = 0; t < NC * NT; ++t) decay_tile(t % NC, t / NC);
                FENCE;
            }
            auto update = [&](int i, int k) __attribute__((always_inline)) {
                const int q = TERMS - 1 - k / NC, n = k % NC;
                S[n][i % NT] = mfma32(yf[i % 3], __builtin_bit_cast(bf16x8, term[i / NT][n][q]), S[n][i % NT]);
            };
            // the first half's update, with the second split; the outputs take the place
            // of the wave's columns of z
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                read_y(i + 2);
#pragma unroll
                for (int k = 0; k < TERMS * NC; ++k) {
                    update(i, k);
                    const int at = i * TERMS * NC + k;  // of TERMS NC NT
                    if (!STATES && at >= 2 * NC && at < 6 * NC) {
                        const int q = (at - 2 * NC) / NC, n = at % NC;
                        *reinterpret_cast<bf16x4*>(zt + o_off[n] + 16 * q * D2) = to_bf16x4(acc[n][q]);
                    } else {
#pragma unroll
                        for (int u = 0; u < 16 * NC; ++u)
                            if (!STATES ? at >= 6 * NC && u * (TERMS * NT - 6) / 16 == at - 6 * NC : u * TERMS * NT / 16 == at)
                                split(1, u);
                    }
                    FENCE;
                }
            }
            // the second, with the rounding of the state for the next chunk
#pragma unroll
            for (int i = NT; i < 2 * NT; ++i) {
                if (i + 2 < 2 * NT) read_y(i + 2);
#pragma unroll
                for (int k = 0; k < TERMS * NC; ++k) {
                    update(i, k);
                    const int done = (i - NT) / 2 - 1;  // tiles 2 done and 2 done + 1 are final
                    if (i % 2 == 1 && done >= 0 && k < NC) round_state(k, done);
                    FENCE;
                }
            }
#pragma unroll
            for (int n = 0; n < NC; ++n) round_state(n, KS - 1);
            settle();
            __syncthreads();
        }
    }

    if (p.s_out && (p.s_out_slots || sg.p1 == sg.len)) {
        float* s = p.s_out + ((int64_t)(p.s_out_slots ? slot : sg.n) * H + h) * (D1 * D2) + state_at;
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int kt = 0; kt < NT; ++kt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[tile_channel(kt, 4 * g + i) * p.row + 16 * n * p.col] = S[n][kt][i];
    }
}

// A workgroup's part of a launch of (heads of a slot x slots, passes): heads fastest,
// then the passes, which read the same rows, then the slots (see wide_grid).
struct Work {
    int pass, slot, h;
    __device__ __forceinline__ explicit Work(int H) {
        const uint32_t id = (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
        h = id % H;
        pass = id / H % gridDim.y;
        slot = id / H / gridDim.y;
    }
};

template <int D1, int D2, int TERMS, bool STATES>
__global__ __launch_bounds__(512, 2) void la_chunk_kernel(LaArgs a) {
    __shared__ __align__(16) unsigned char lds[lds_bytes<D1, D2, STATES>()];
    const Work w(a.s.H);
    if (w.slot >= a.s.n_slots) return;
    chunk_pass<D1, D2, TERMS, STATES>(a, a.pass[w.pass], w.slot, w.h, lds);
}

// passes over 64 x 128 and 128 x 64 states side by side
template <int TERMS>
__global__ __launch_bounds__(512, 2) void la_chunk_mixed_kernel(LaArgs a) {
    constexpr int A = lds_bytes<64, 128, false>(), B = lds_bytes<128, 64, false>();
    __shared__ __align__(16) unsigned char lds[A > B ? A : B];
    const Work w(a.s.H);
    if (w.slot >= a.s.n_slots) return;
    const LaPass& p = a.pass[w.pass];
    if (p.D2 == 128) chunk_pass<64, 128, TERMS, false>(a, p, w.slot, w.h, lds);
    else chunk_pass<128, 64, TERMS, false>(a, p, w.slot, w.h, lds);
}

// Entering states of the segments: for a sequence's segments in order,
// E_0 = the sequence's own entering state, E_(s+1) = a^seg_tokens E_s + U_s,
// written over U.  One thread per four elements of a (sequence, head)'s state.
__global__ __launch_bounds__(256) void la_scan_kernel(LaScanArgs a) {
    const int dir = blockIdx.y;
    const int per = a.elems / 1024;  // workgroups per state (K V is a multiple of 4096)
    const uint32_t wg = blockIdx.z * gridDim.x + blockIdx.x;
    const int pair = wg / per, n = pair / a.s.H, h = pair % a.s.H;
    if (n >= a.s.n_seqs) return;
    const int e = (int)(wg % per * 256 + threadIdx.x) * 4;
    int slot, len;
    if (!a.s.cu) {
        slot = n * a.s.seg_per_seq;
        len = a.s.T;
    } else {
        const int t0 = clamp_tok(a.s, a.s.cu[n]);
        slot = t0 / a.s.seg_tokens + n;
        len = max(clamp_tok(a.s, a.s.cu[n + 1]) - t0, 0);
    }
    const int segs = max(1, (len + a.s.seg_tokens - 1) / a.s.seg_tokens);
    const float ld = head_log_decay(a.log_decay, h);
    const float x = ld * (float)a.s.seg_tokens;
    const bool near = x > -0.6f;
    const float c0 = near ? 1.f : 0.f, c1 = near ? expm1f(x) : expf(x);
    floatx4 s = {0.f, 0.f, 0.f, 0.f};
    if (a.init[dir]) s = *reinterpret_cast<const floatx4*>(a.init[dir] + ((int64_t)n * a.s.H + h) * a.elems + e);
    for (int i = 0; i < segs && slot + i < a.s.n_slots; ++i) {
        floatx4* w = reinterpret_cast<floatx4*>(a.state[dir] + ((int64_t)(slot + i) * a.s.H + h) * a.elems + e);
        const floatx4 u = i + 1 < segs ? *w : floatx4{0.f, 0.f, 0.f, 0.f};
        *w = s;
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = fmaf(s[j], c1, s[j] * c0) + u[j];
    }
}

void launch_la_chunk(const LaArgs& a, int n, bool states, hipStream_t stream) {
    int terms = 2;
    bool mixed = false;
    for (int i = 0; i < n; ++i) {
        if (a.pass[i].s_out) terms = 3;
        mixed |= a.pass[i].D1 != a.pass[0].D1;
    }
    const dim3 grid = wide_grid((int64_t)a.s.n_slots * a.s.H, 512, (unsigned)n);
    if (mixed) {
        if (terms == 3) hipLaunchKernelGGL((la_chunk_mixed_kernel<3>), grid, dim3(512), 0, stream, a);
        else hipLaunchKernelGGL((la_chunk_mixed_kernel<2>), grid, dim3(512), 0, stream, a);
        return;
    }
    auto go = [&](auto d1, auto d2) {
        constexpr int X = decltype(d1)::value, Z = decltype(d2)::value;
        if (states) hipLaunchKernelGGL((la_chunk_kernel<X, Z, 3, true>), grid, dim3(512), 0, stream, a);
        else if (terms == 3) hipLaunchKernelGGL((la_chunk_kernel<X, Z, 3, false>), grid, dim3(512), 0, stream, a);
        else hipLaunchKernelGGL((la_chunk_kernel<X, Z, 2, false>), grid, dim3(512), 0, stream, a);
    };
    const std::integral_constant<int, 64> s{};
    const std::integral_constant<int, 128> l{};
    const int D1 = a.pass[0].D1, D2 = a.pass[0].D2;
    if (D1 == 128 && D2 == 128) go(l, l);
    else if (D1 == 128) go(l, s);
    else if (D2 == 128) go(s, l);
    else go(s, s);
}

void launch_la_scan(const LaScanArgs& a, hipStream_t stream) {
    const dim3 grid = wide_grid((int64_t)a.s.n_seqs * a.s.H * (a.elems / 1024), 256, (unsigned)a.n_dirs);
    hipLaunchKernelGGL(la_scan_kernel, grid, dim3(256), 0, stream, a);
}

}  // namespace kda
