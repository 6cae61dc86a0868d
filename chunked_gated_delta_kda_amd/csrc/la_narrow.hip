// la_narrow.hip -- chunked linear attention for few (sequence, head) pairs (gfx950):
// the passes of la_chunk.hip (its mathematics and precision) over whole sequences, in
// workgroups of 32 state columns.  A decayed z always has three terms here; la_chunk.hip
// takes two in launches that return no state.  With a state returned the two give the
// same bits, without one outputs differ by the third term, below 2^-15 of a summand
// before they are rounded to bf16.
//
// One workgroup per (sequence, head, 32 columns); the column blocks of one head are
// neighbours on one XCD, whose L2 serves the rows of x and y to all of them.  Eight
// waves in two roles, side by side on every SIMD:
//  - four output waves, 16 queries each: P^T of their queries from the x rows in their
//    registers and the y tile in LDS (its D layout is the operand of the product with
//    z, so P stays in registers), plus S^T x from the bf16 copy of S in LDS; they also
//    load z and leave it in LDS, raw and as the decayed terms of the update;
//  - four state waves, half the D1 rows and 16 columns each: y into LDS, the update,
//    and the copy of S for the next chunk.
// One barrier a chunk; y, z and the copy are double-buffered, rows are loaded three
// chunks ahead.
//
// What bounds it: the way it reads.  A column block reads z in 64-byte pieces and x
// and y once per block through L2: 2 x 2048 tokens, 32 heads of 128 x 128 (134 MB)
// take 44 to 48 us, 2.8 to 3.0 TB/s, with or without the products; the products alone
// 35 us.  With few workgroups it is the chain within a chunk, 1.0 to 1.3 us: 256 tokens,
// 4 heads of 64 x 64, take 6.0 us where la_chunk.hip takes 8.5.
#include "la_device.h"

namespace kda {

constexpr int LA_COLS = 32;  // state columns per workgroup

constexpr int narrow_lds_bytes(int D1) { return 2 * LC * D1 * 2 + 2 * 4 * LC * LA_COLS * 2 + 2 * 2 * (D1 / 32) * 64 * 16; }

template <int D1>
__device__ __forceinline__ void narrow_pass(const LaArgs& a, const LaPass& p, unsigned char* lds) {
    constexpr int KS = D1 / 32;       // 16x16x32 steps over D1
    constexpr int NT = D1 / 32;       // state tiles of a wave (half of D1 / 16)
    constexpr int YV = D1 / 32;       // 16-byte pieces of the y tile per thread of its four waves
    constexpr int TPR = D1 / 8;       // threads per row of the y tile
    constexpr int YROWS = 256 / TPR;  // rows they cover at once
    bf16(*const ytile)[LC * D1] = reinterpret_cast<bf16(*)[LC * D1]>(lds);
    bf16(*const ztile)[LC * LA_COLS] = reinterpret_cast<bf16(*)[LC * LA_COLS]>(ytile + 2);
    bf16(*const zterm)[3][LC * LA_COLS] = reinterpret_cast<bf16(*)[3][LC * LA_COLS]>(ztile + 2);
    u32x4(*const scopy)[2][KS][64] = reinterpret_cast<u32x4(*)[2][KS][64]>(zterm + 2);

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

    const int tid = threadIdx.x & 255;  // within the four waves of a role
    const int lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool out_role = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) == 0;
    const int D2 = p.D2, c0 = cb * LA_COLS;
    const int late = p.reverse ? 1 : 0;

    if (a.s.cu && (sg.n == 0 || sg.n == a.s.n_seqs - 1)) {
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

    // z of a chunk, in 16-byte pieces, left in LDS as it is and, decayed to the
    // chunk's end, as three bf16 terms
    const uint16_t* const zrow = p.z + (tok0 * H + h) * D2 + c0 + 8 * (lane & 3);
    auto load_z = [&](int c, int row) { return *reinterpret_cast<const u32x4*>(zrow + at(c, row) * zstep); };
    auto weight = [&](int n, int row) { return row < n ? exp2_hw((n - 1 - row + late) * l2) * p.z_scale : 0.f; };
    auto put_z = [&](int c, int row, float full, u32x4 raw) __attribute__((always_inline)) {
        const int n = np - c * LC;
        float wt = full;
        if (n < LC) wt = weight(n, row);
        u32x4 term[3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v0 = decayed(bf_lo(raw[e]), wt), v1 = decayed(bf_hi(raw[e]), wt);
#pragma unroll
            for (int q = 0; q < 3; ++q) term[q][e] = take_term(v0, v1);
        }
        const int at = row * LA_COLS + 8 * (lane & 3);
        *reinterpret_cast<u32x4*>(&ztile[c & 1][at]) = raw;
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<u32x4*>(&zterm[c & 1][q][at]) = term[q];
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

            // rows of z that this wave stages: 32, 16, 16 and none, since the waves have
            // one, two, three and four tiles of P
            constexpr int ZN = W == 0 ? 2 : W == 3 ? 0 : 1, Z0 = W == 0 ? 0 : 16 * (W + 1);
            const int zr = Z0 + (lane >> 2);
            const float z_full0 = weight(LC, zr), z_full1 = weight(LC, zr + 16);
            u32x4 xs[2][KS], zs[2][ZN + (ZN == 0)];
            auto load_zs = [&](int c, u32x4 (&z)[ZN + (ZN == 0)]) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < ZN; ++i) z[i] = load_z(c, zr + 16 * i);
            };
            auto put_zs = [&](int c, const u32x4 (&z)[ZN + (ZN == 0)]) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < ZN; ++i) put_z(c, zr + 16 * i, i ? z_full1 : z_full0, z[i]);
            };
            auto load_x = [&](int c, u32x4 (&x)[KS]) __attribute__((always_inline)) {
                const uint16_t* q = xrow + at(c, i0) * ystep;
#pragma unroll
                for (int j = 0; j < KS; ++j) x[j] = *reinterpret_cast<const u32x4*>(q + 32 * j);
            };
            {
                u32x4 z0[ZN + (ZN == 0)];
                load_zs(0, z0);
                load_x(0, xs[0]);
                load_zs(1, zs[1]);
                load_x(1, xs[1]);
                load_zs(2, zs[0]);
                put_zs(0, z0);
            }
            __syncthreads();
            // chunk c from x; z holds chunk c + 1, and takes chunk c + 3
            auto chunk = [&](int c, u32x4 (&x)[KS], u32x4 (&z)[ZN + (ZN == 0)], auto full) __attribute__((always_inline)) {
                const int buf = c & 1;
                const bf16* yt = ytile[buf];
                const bf16* zt = ztile[buf] + zt_off;
                if (c + 1 < nc) put_zs(c + 1, z);
                load_zs(c + 3, z);
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
                for (int k = 0; k <= W; k += 2)
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) {
                        const bf16* z0 = zt + 16 * k * LA_COLS + 4 * ct;
                        acc[ct] = mfma32(join(read_t(z0), k < W ? read_t(z0 + 16 * LA_COLS) : none),
                                         join(pf[W - k], k < W ? pf[W - k - (k < W)] : none), acc[ct]);
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
        const float* s = p.s_in + ((int64_t)sg.n * H + h) * sz + (int64_t)scol * p.col;
        auto load = [&](int row) __attribute__((always_inline)) {
#pragma unroll
            for (int kt = 0; kt < NT; ++kt) S[kt] = load_state(s, tile_channel(kh * NT + kt, 4 * g), row);
        };
        if (p.row == 1) load(1);
        else load(p.row);
    } else {
#pragma unroll
        for (int kt = 0; kt < NT; ++kt) S[kt] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
    if (nc > 0) {
        ChunkDecay chunk_decay(ld);
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
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                const bf16x8 f = join(to_bf16x4(S[2 * j]), to_bf16x4(S[2 * j + 1]));
                scopy[buf][vh][kh * (NT / 2) + j][lane] = __builtin_bit_cast(u32x4, f);
            }
        };
        int yt_off[NT / 2];  // transposing reads of y, tiles 2 T and 2 T + 1 of this wave
#pragma unroll
        for (int j = 0; j < NT / 2; ++j)
            yt_off[j] = (4 * g + (r >> 2)) * D1 + 8 * ((4 * (kh * (NT / 2) + j) + (r & 3)) ^ swizzle<D1>(4 * g + (r >> 2)));

        u32x4 ys[2][YV];
        {
            u32x4 y0[YV];
            load_y(0, y0);
            load_y(1, ys[1]);
            load_y(2, ys[0]);
            put_y(0, y0);
            put_s(0);
        }
        __syncthreads();
        // chunk c; y holds chunk c + 1, and takes chunk c + 3
        auto chunk = [&](int c, u32x4 (&y)[YV]) __attribute__((always_inline)) {
            const int buf = c & 1;
            if (c + 1 < nc) put_y(c + 1, y);
            load_y(c + 3, y);
            const int n = np - c * LC;
            float decay = chunk_decay.step();
            if (n < LC) decay = exp2_hw(n * l2);
#pragma unroll
            for (int kt = 0; kt < NT; ++kt) S[kt] *= decay;
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
            settle();
            if (c + 1 < nc) {
                put_s(buf ^ 1);
                __syncthreads();
            }
        };
        int c = 0;
        for (; c + 1 < nc; c += 2) {
            chunk(c, ys[1]);
            chunk(c + 1, ys[0]);
        }
        if (c < nc) chunk(c, ys[1]);
    }

    if (p.s_out) {
        float* s = p.s_out + ((int64_t)sg.n * H + h) * sz + (int64_t)scol * p.col;
#pragma unroll
        for (int kt = 0; kt < NT; ++kt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[tile_channel(kh * NT + kt, 4 * g + i) * p.row] = S[kt][i];
    }
}

// (128-row and 64-row states, side by side where a batch has both)
template <bool MIXED, int D1>
__global__ __launch_bounds__(512, 4) void la_narrow_kernel(LaArgs a) {
    __shared__ __align__(16) unsigned char lds[narrow_lds_bytes(MIXED ? 128 : D1)];
    const LaPass& p = a.pass[blockIdx.y];
    if (MIXED && p.D1 == 64) narrow_pass<64>(a, p, lds);
    else narrow_pass<D1>(a, p, lds);
}

int64_t la_narrow_groups(int64_t pairs, int cols) { return (pairs + 7) / 8 * 8 * (cols / LA_COLS); }

void launch_la_narrow(const LaArgs& a, int n, hipStream_t stream) {
    int cols = 64;
    bool mixed = false;
    for (int i = 0; i < n; ++i) {
        cols = a.pass[i].D2 > cols ? a.pass[i].D2 : cols;
        mixed |= a.pass[i].D1 != a.pass[0].D1;
    }
    const dim3 grid((unsigned)la_narrow_groups((int64_t)a.s.n_seqs * a.s.H, cols), (unsigned)n);
    if (mixed) hipLaunchKernelGGL((la_narrow_kernel<true, 128>), grid, dim3(512), 0, stream, a);
    else if (a.pass[0].D1 == 128) hipLaunchKernelGGL((la_narrow_kernel<false, 128>), grid, dim3(512), 0, stream, a);
    else hipLaunchKernelGGL((la_narrow_kernel<false, 64>), grid, dim3(512), 0, stream, a);
}

}  // namespace kda
