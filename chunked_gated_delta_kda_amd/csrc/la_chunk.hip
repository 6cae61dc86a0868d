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
// One workgroup of four waves per (segment, head, 32 state columns); the
// column blocks of one head are neighbours on one XCD, whose L2 serves the
// rows of x and y to all of them.  Per chunk, wave w
//  - forms P^T for its 16 queries (key tiles 0..w; 16x16x32 MFMAs on the raw
//    bf16 rows), whose D layout is the operand of the product with z, so P
//    stays in registers; decays are a table of 16 values a lane;
//  - adds S^T x from the bf16 copy of S that the waves left in LDS;
//  - updates its quarter of S (half of the D1 rows, 16 columns) in fp32
//    accumulators, and leaves its bf16 copy for the next chunk.
// One barrier a chunk: the y and z tiles and the copy of S are double-buffered.
//
// Precision: raw bf16 operands; P and the copy of S are rounded to bf16 once
// each (outputs are bf16).  The state itself is fp32 to its last bits, since
// it is returned: a token's decayed z is split into three bf16 terms (24
// bits), so every product of the update is exact, and the decay of a chunk is
// applied as S + (a^n - 1) S where a^n is near one, or the rounding of a^n
// would add up over thousands of chunks.
#include "kda_common.h"
#include "la_launch.h"

namespace kda {

namespace {

constexpr int LC = LA_CHUNK;

// the type's lowest log decay that matters: exp(-200) is zero in fp32 twice over
constexpr float LOG_DECAY_FLOOR = -200.f;

__device__ __forceinline__ float head_log_decay(const float* p, int h) {
    const float v = p[h];
    return v < LOG_DECAY_FLOOR ? LOG_DECAY_FLOOR : v;  // keeps a NaN
}

// a segment: tokens t0 .. t0 + len of sequence n, positions p0 .. p1
struct Seg {
    int n;
    int t0, len;
    int p0, p1;
};

__device__ __forceinline__ int clamp_tok(const LaSeqs& s, int v) { return min(max(v, 0), s.T); }

// The segment of a slot; false if the slot holds none.  Offsets are clamped
// to the batch, so an array that is not what it should be gives wrong
// results, never an access out of bounds.
__device__ __forceinline__ bool find_seg(const LaSeqs& s, int slot, Seg& g) {
    int seg;
    if (!s.cu) {
        g.n = slot / s.seg_per_seq;
        seg = slot % s.seg_per_seq;
        g.t0 = g.n * s.T;
        g.len = s.T;
    } else {
        int n = slot;
        seg = 0;
        if (s.seg_tokens) {
            // the last sequence whose first slot is not behind this one: 64
            // candidates at a time
            const int lane = threadIdx.x & 63;
            int lo = 0, cnt = s.n_seqs;
            for (;;) {
                const int step = (cnt + 63) / 64;
                const int i = lo + lane * step;
                const bool le = lane * step < cnt &&
                                clamp_tok(s, s.cu[min(i, s.n_seqs)]) / s.seg_tokens + i <= slot;
                const int k = __popcll(__ballot(le)) - 1;
                if (k < 0) return false;
                lo += k * step;
                if (step == 1) break;
                cnt = min(step, cnt - k * step);
            }
            n = lo;
            seg = slot - (clamp_tok(s, s.cu[n]) / s.seg_tokens + n);
        }
        g.n = n;
        g.t0 = clamp_tok(s, s.cu[n]);
        g.len = max(clamp_tok(s, s.cu[n + 1]) - g.t0, 0);
    }
    if (!s.seg_tokens) {
        g.p0 = 0;
        g.p1 = g.len;
        return true;
    }
    if (seg > 0 && (int64_t)seg * s.seg_tokens >= g.len) return false;
    g.p0 = seg * s.seg_tokens;
    g.p1 = g.p0 + min(g.len - g.p0, s.seg_tokens);
    return true;
}

// Row r of tile t of the state (and of an operand that contracts over the
// chunk's tokens): channel 32 (t / 2) + 8 (r / 4) + 4 (t % 2) + r % 4, so the
// accumulators of tiles 2j and 2j+1 are the eight channels 32 j + 8 g + e of
// the operand of a product that contracts over them.

// Operand that contracts over tokens: lane (r, g) receives rows 4 g .. 4 g + 3,
// column channel(t, r) of 16 rows of an LDS tile, by one transposing read
// (ds_read_b64_tr_b16): in each group of 16 lanes, lane r fetches four
// consecutive columns of row 4 g + r / 4, those that lanes 4 (r % 4) .. + 3
// receive.
__device__ __forceinline__ bf16x4 read_t(const bf16* p) {
    typedef __attribute__((address_space(3))) short4_t* lds_short4;
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4)p));
}

__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The y tile holds its rows without padding (two workgroups of 80 KB share a
// CU's LDS); 16-byte unit u of row m sits at unit u ^ swizzle(m).  Sixteen rows
// of one unit (the P products) then lie in sixteen different units, and the
// four rows of a transposing read in four different 64-byte blocks.
template <int D1>
__device__ __forceinline__ int swizzle(int m) {
    return D1 == 128 ? 4 * (m & 3) + ((m >> 2) & 3) : 4 * ((m >> 1) & 1) + ((m >> 2) & 3);
}

}  // namespace

template <int D1, bool STATES>
__global__ __launch_bounds__(STATES ? 256 : 512, STATES ? 2 : 4) void la_chunk_kernel(LaArgs a) {
    constexpr int KS = D1 / 32;       // 16x16x32 steps over D1
    constexpr int NT = D1 / 32;       // state tiles of a wave (half of D1 / 16)
    constexpr int YV = D1 / 32;       // 16-byte pieces of the y tile per thread of its four waves
    constexpr int TPR = D1 / 8;       // threads per row of the y tile
    constexpr int YROWS = 256 / TPR;  // rows they cover at once
    __shared__ __align__(16) bf16 ytile[2][LC * D1];
    __shared__ __align__(16) bf16 ztile[STATES ? 1 : 2][LC * LA_COLS];
    __shared__ __align__(16) bf16 zterm[2][3][LC * LA_COLS];
    __shared__ u32x4 scopy[STATES ? 1 : 2][2][STATES ? 1 : KS][64];

    const LaPass& p = a.pass[blockIdx.y];
    const int H = a.s.H;
    const int ncb = p.D2 / LA_COLS;
    // workgroups are dealt to the eight XCDs in turn: the column blocks of one
    // (segment, head) follow each other on one of them
    const int64_t b = blockIdx.x;
    const int64_t group = (b / 8 / ncb) * 8 + b % 8;
    const int cb = (int)(b / 8 % ncb);
    if (group >= (int64_t)a.s.n_slots * H) return;
    const int slot = (int)(group / H), h = (int)(group % H);
    Seg sg;
    if (!find_seg(a.s, slot, sg)) return;
    if (STATES && sg.p1 == sg.len) return;  // nobody enters from a sequence's last segment

    const int tid = threadIdx.x & 255;  // within the four waves of a role
    const int lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool out_role = !STATES && __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) == 0;
    const int D2 = p.D2, c0 = cb * LA_COLS;
    const int late = p.reverse ? 1 : 0;

    if (!STATES && a.s.cu && sg.p0 == 0 && (sg.n == 0 || sg.n == a.s.n_seqs - 1)) {
        // rows outside every sequence: zeros
        auto zero_rows = [&](int lo, int hi) {
            for (int t = lo + ((int)threadIdx.x >> 2); t < hi; t += 128)
                *reinterpret_cast<u32x4*>(p.o + ((int64_t)t * H + h) * D2 + c0 + 8 * (tid & 3)) = u32x4{0, 0, 0, 0};
        };
        if (sg.n == 0) zero_rows(0, sg.t0);
        if (sg.n == a.s.n_seqs - 1) zero_rows(sg.t0 + sg.len, a.s.T);
    }

    const float ld = head_log_decay(a.log_decay, h);
    const float l2 = ld * LOG2E;

    // ---- rows of x, y, z at a position.  Positions behind the segment's end
    // read its last row, whose weight in the state is then zero and whose
    // output is not stored: every load is unconditional.
    const int np = sg.p1 - sg.p0, nc = (np + LC - 1) / LC;
    const int64_t step = p.reverse ? -1 : 1;
    const int64_t tok0 = p.reverse ? (int64_t)sg.t0 + sg.len - 1 - sg.p0 : (int64_t)sg.t0 + sg.p0;
    const int64_t ystep = step * H * D1, zstep = step * H * D2;
    auto at = [&](int c, int row) { return (int64_t)min(c * LC + row, np - 1); };

    // z of a chunk: one 16-byte piece a thread, left in LDS as it is and, decayed
    // to the chunk's end, as three bf16 terms
    const uint16_t* const zrow = p.z + (tok0 * H + h) * D2 + c0 + 8 * (tid & 3);
    auto load_z = [&](int c) { return *reinterpret_cast<const u32x4*>(zrow + at(c, tid >> 2) * zstep); };
    const float z_full = exp2_hw((LC - 1 - (tid >> 2) + late) * l2) * p.z_scale;
    auto put_z = [&](int c, u32x4 raw) {
        const int n = np - c * LC, row = tid >> 2;
        float wt = z_full;
        if (n < LC) wt = row < n ? exp2_hw((n - 1 - row + late) * l2) * p.z_scale : 0.f;
        const bf16x8 z = __builtin_bit_cast(bf16x8, raw);
        bf16x8 term[3];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = (float)z[e] * wt;
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                term[q][e] = (bf16)v;
                v -= (float)term[q][e];
            }
        }
        if constexpr (!STATES) *reinterpret_cast<u32x4*>(&ztile[c & 1][8 * tid]) = raw;
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<bf16x8*>(&zterm[c & 1][q][8 * tid]) = term[q];
    };
    // where a transposing read of a z tile starts (tile ct of 16 columns: + 4 ct)
    const int zt_off = (4 * g + (r >> 2)) * LA_COLS + 8 * (r & 3);

    if (out_role) {
        if (nc == 0) return;
        // ================= outputs: wave w owns the chunk's queries 16 w + r
        auto outputs = [&](auto wc) __attribute__((always_inline)) {
            constexpr int W = decltype(wc)::value;
            const int i0 = 16 * W + r;
            const uint16_t* const xrow = p.x + (tok0 * H + h) * D1 + 8 * g;
            uint16_t* const orow = p.o + (tok0 * H + h) * D2 + c0 + 8 * g;
            const float up = exp2_hw((i0 + 1 - late) * l2) * p.x_scale;
            float dec[W + 1][4];  // decay from key 16 (W - d) + 4 g + i
#pragma unroll
            for (int d = 0; d <= W; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) dec[d][i] = exp2_hw(max(16 * d + r - 4 * g - i, 0) * l2) * p.in_scale;
            int koff[KS];
#pragma unroll
            for (int j = 0; j < KS; ++j) koff[j] = r * D1 + 8 * ((4 * j + g) ^ swizzle<D1>(r));

            u32x4 xs[2][KS], zs[2];
            auto load_x = [&](int c, u32x4 (&x)[KS]) __attribute__((always_inline)) {
                const uint16_t* q = xrow + at(c, i0) * ystep;
#pragma unroll
                for (int j = 0; j < KS; ++j) x[j] = *reinterpret_cast<const u32x4*>(q + 32 * j);
            };
            {
                const u32x4 z0 = load_z(0);
                load_x(0, xs[0]);
                zs[1] = load_z(1);
                load_x(1, xs[1]);
                zs[0] = load_z(2);
                put_z(0, z0);
            }
            __syncthreads();
            // chunk c from x; z holds chunk c + 1, and takes chunk c + 3
            auto chunk = [&](int c, u32x4 (&x)[KS], u32x4& z, auto full) __attribute__((always_inline)) {
                const int buf = c & 1;
                const bf16* yt = ytile[buf];
                const bf16* zt = ztile[buf] + zt_off;
                if (c + 1 < nc) put_z(c + 1, z);
                z = load_z(c + 3);
                // S^T x: D rows are the columns channel(ct, .), D columns the queries
                floatx4 acc[2];
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) {
                    acc[ct] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < KS; ++j)
                        acc[ct] = mfma32(__builtin_bit_cast(bf16x8, scopy[buf][ct][j][lane]), __builtin_bit_cast(bf16x8, x[j]), acc[ct]);
                }
                // P^T of the key tiles W, W - 1, ...
                floatx4 pt[W + 1];
#pragma unroll
                for (int d = 0; d <= W; ++d) {
                    pt[d] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < KS; ++j)
                        pt[d] = mfma32(*reinterpret_cast<const bf16x8*>(yt + 16 * (W - d) * D1 + koff[j]), __builtin_bit_cast(bf16x8, x[j]), pt[d]);
                }
                load_x(c + 2, x);
                acc[0] *= up;
                acc[1] *= up;
                bf16x4 pf[W + 1];
#pragma unroll
                for (int d = 0; d <= W; ++d) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        pt[d][i] *= dec[d][i];
                        if (d == 0 && r < 4 * g + i) pt[d][i] = 0.f;
                    }
                    pf[d] = to_bf16x4(pt[d]);
                }
                // (P z), two key tiles at a time; a last odd one is padded with zeros.
                // (Not by a 16x16x16 product: issued right behind the 16x16x32 one
                // whose result it adds to, it read two stale accumulators now and then.)
                const bf16x4 none = {};
#pragma unroll
                for (int d = 0; d <= W; d += 2)
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) {
                        const bf16* z0 = zt + 16 * (W - d) * LA_COLS + 4 * ct;
                        acc[ct] = mfma32(join(read_t(z0), d < W ? read_t(z0 - 16 * LA_COLS) : none),
                                         join(pf[d], d < W ? pf[d < W ? d + 1 : d] : none), acc[ct]);
                    }
                const u32x4 ov = __builtin_bit_cast(u32x4, join(to_bf16x4(acc[0]), to_bf16x4(acc[1])));
                uint16_t* o = orow + at(c, i0) * zstep;
                if (decltype(full)::value || c * LC + i0 < np) *reinterpret_cast<u32x4*>(o) = ov;
                if (c + 1 < nc) __syncthreads();
            };
            const int nf = np / LC;  // full chunks
            int c = 0;
            for (; c + 1 < nf; c += 2) {
                chunk(c, xs[0], zs[1], std::true_type{});
                chunk(c + 1, xs[1], zs[0], std::true_type{});
            }
            if (c < nf) {
                chunk(c, xs[0], zs[1], std::true_type{});
                if (nf < nc) chunk(c + 1, xs[1], zs[0], std::false_type{});
            } else if (nf < nc) {
                chunk(c, xs[0], zs[1], std::false_type{});
            }
        };
        if (w == 0) outputs(std::integral_constant<int, 0>{});
        else if (w == 1) outputs(std::integral_constant<int, 1>{});
        else if (w == 2) outputs(std::integral_constant<int, 2>{});
        else outputs(std::integral_constant<int, 3>{});
        return;
    }

    // ================= the state: wave w owns half the D1 rows and 16 columns.
    // Accumulator element i of tile kt is row channel(kh NT + kt, 4 g + i),
    // column c0 + channel(vh, r).
    const int kh = w >> 1, vh = w & 1;
    floatx4 S[NT];
    const int64_t sz = (int64_t)D1 * D2;
    const int scol = c0 + tile_channel(vh, r);
    if (p.s_in) {
        const float* s = p.s_in + ((int64_t)(p.s_in_slots ? slot : sg.n) * H + h) * sz + (int64_t)scol * p.col;
#pragma unroll
        for (int kt = 0; kt < NT; ++kt)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[kt][i] = s[tile_channel(kh * NT + kt, 4 * g + i) * p.row];
    } else {
#pragma unroll
        for (int kt = 0; kt < NT; ++kt) S[kt] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
    if (nc > 0) {
        float c_s0, c_s1;  // a chunk's decay, as c_s0 S + c_s1 S
        auto set_decay = [&](int n) {
            const float x = n * ld;
            const bool near = x > -0.6f;
            c_s0 = near ? 1.f : 0.f;
            c_s1 = near ? expm1f(x) : exp2_hw(n * l2);
        };
        const uint16_t* const yrow = p.y + (tok0 * H + h) * D1 + 8 * (tid % TPR);
        bf16* const yput = &ytile[0][(tid / TPR) * D1 + 8 * ((tid % TPR) ^ swizzle<D1>(tid / TPR))];
        auto load_y = [&](int c, u32x4 (&y)[YV]) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < YV; ++i) y[i] = *reinterpret_cast<const u32x4*>(yrow + at(c, tid / TPR + i * YROWS) * ystep);
        };
        auto put_y = [&](int c, const u32x4 (&y)[YV]) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < YV; ++i) *reinterpret_cast<u32x4*>(yput + (c & 1) * LC * D1 + i * YROWS * D1) = y[i];
        };
        auto put_s = [&](int buf) __attribute__((always_inline)) {
            if constexpr (!STATES) {
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    const bf16x8 f = join(to_bf16x4(S[2 * j]), to_bf16x4(S[2 * j + 1]));
                    scopy[buf][vh][kh * (NT / 2) + j][lane] = __builtin_bit_cast(u32x4, f);
                }
            }
        };
        int yt_off[NT / 2];  // transposing reads of y, tiles 2 T and 2 T + 1 of this wave
#pragma unroll
        for (int j = 0; j < NT / 2; ++j)
            yt_off[j] = (4 * g + (r >> 2)) * D1 + 8 * ((4 * (kh * (NT / 2) + j) + (r & 3)) ^ swizzle<D1>(4 * g + (r >> 2)));

        u32x4 ys[2][YV], zs[2];
        {
            u32x4 y0[YV];
            load_y(0, y0);
            u32x4 z0;
            if constexpr (STATES) z0 = load_z(0);
            load_y(1, ys[1]);
            if constexpr (STATES) zs[1] = load_z(1);
            load_y(2, ys[0]);
            if constexpr (STATES) zs[0] = load_z(2);
            set_decay(min(np, LC));
            put_y(0, y0);
            if constexpr (STATES) put_z(0, z0);
            put_s(0);
        }
        __syncthreads();
        // chunk c; y (and z) hold chunk c + 1, and take chunk c + 3
        auto chunk = [&](int c, u32x4 (&y)[YV], u32x4& z) __attribute__((always_inline)) {
            const int buf = c & 1;
            if (c + 1 < nc) {
                put_y(c + 1, y);
                if constexpr (STATES) put_z(c + 1, z);
            }
            load_y(c + 3, y);
            if constexpr (STATES) z = load_z(c + 3);
            const int n = np - c * LC;
            if (n < LC && c > 0) set_decay(n);
#pragma unroll
            for (int kt = 0; kt < NT; ++kt)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[kt][i] = fmaf(S[kt][i], c_s1, S[kt][i] * c_s0);
            const bf16* yt = ytile[buf];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                bf16x8 z3[3];
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    const bf16* z0 = zterm[buf][q] + 32 * m * LA_COLS + zt_off + 4 * vh;
                    z3[q] = join(read_t(z0), read_t(z0 + 16 * LA_COLS));
                }
#pragma unroll
                for (int kt = 0; kt < NT; ++kt) {
                    const bf16* y0 = yt + 32 * m * D1 + yt_off[kt / 2] + 4 * (kt & 1);
                    const bf16x8 yf = join(read_t(y0), read_t(y0 + 16 * D1));
#pragma unroll
                    for (int q = 2; q >= 0; --q) S[kt] = mfma32(yf, z3[q], S[kt]);
                }
            }
            if (c + 1 < nc) {
                put_s(buf ^ 1);
                __syncthreads();
            }
        };
        int c = 0;
        for (; c + 1 < nc; c += 2) {
            chunk(c, ys[1], zs[1]);
            chunk(c + 1, ys[0], zs[0]);
        }
        if (c < nc) chunk(c, ys[1], zs[1]);
    }

    if (p.s_out && (p.s_out_slots || sg.p1 == sg.len)) {
        float* s = p.s_out + ((int64_t)(p.s_out_slots ? slot : sg.n) * H + h) * sz + (int64_t)scol * p.col;
#pragma unroll
        for (int kt = 0; kt < NT; ++kt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[tile_channel(kh * NT + kt, 4 * g + i) * p.row] = S[kt][i];
    }
}

// Entering states of the segments: for a sequence's segments in order,
// E_0 = the sequence's own entering state, E_(s+1) = a^seg_tokens E_s + U_s,
// written over U.  One thread per four elements of a (sequence, head)'s state.
__global__ __launch_bounds__(256) void la_scan_kernel(LaScanArgs a) {
    const int dir = blockIdx.y;
    const int per = a.elems / 1024;  // workgroups per state (K V is a multiple of 4096)
    const int pair = blockIdx.x / per, n = pair / a.s.H, h = pair % a.s.H;
    const int e = (int)(blockIdx.x % per * 256 + threadIdx.x) * 4;
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

void launch_la_chunk(const LaArgs& a, int n, int D1, bool states, hipStream_t stream) {
    const int64_t groups = (int64_t)a.s.n_slots * a.s.H;
    int ncb = 0;
    for (int i = 0; i < n; ++i) ncb = max(ncb, a.pass[i].D2 / LA_COLS);
    const dim3 grid((unsigned)((groups + 7) / 8 * 8 * ncb), (unsigned)n);
    if (D1 == 128) {
        if (states) hipLaunchKernelGGL((la_chunk_kernel<128, true>), grid, dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((la_chunk_kernel<128, false>), grid, dim3(512), 0, stream, a);
    } else {
        if (states) hipLaunchKernelGGL((la_chunk_kernel<64, true>), grid, dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((la_chunk_kernel<64, false>), grid, dim3(512), 0, stream, a);
    }
}

void launch_la_scan(const LaScanArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.s.n_seqs * a.s.H * (a.elems / 1024)), (unsigned)a.n_dirs);
    hipLaunchKernelGGL(la_scan_kernel, grid, dim3(256), 0, stream, a);
}

}  // namespace kda
