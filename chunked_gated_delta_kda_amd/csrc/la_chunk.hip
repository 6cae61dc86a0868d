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

constexpr int LA_THREADS = 256;
constexpr int LC = LA_CHUNK;
constexpr int ZS = LA_COLS + 16;  // z tile's row stride: 24 banks on, so four rows do not collide

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
// Operand that contracts over tokens: lane (r, g) holds rows 4 g .. 4 g + 3 of
// the 16 rows at `rows`, column channel(t, r).
__device__ __forceinline__ bf16x4 tile_t(const bf16* rows, int stride, int t, int lane) {
    const int r = lane & 15, g = lane >> 4;
    const bf16* p = rows + 4 * g * stride + tile_channel(t, r);
    return bf16x4{p[0], p[stride], p[2 * stride], p[3 * stride]};
}

__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

}  // namespace

template <int D1, bool STATES>
__global__ __launch_bounds__(LA_THREADS, 2) void la_chunk_kernel(LaArgs a) {
    constexpr int KS = D1 / 32;       // 16x16x32 steps over D1
    constexpr int NT = D1 / 32;       // state tiles of a wave (half of D1 / 16)
    constexpr int YS = D1 + 16;       // y tile's row stride
    constexpr int YV = D1 / 32;       // 16-byte pieces of the y tile per thread
    constexpr int TPR = D1 / 8;       // threads per row of the y tile
    __shared__ __align__(16) bf16 ytile[2][LC][YS];
    __shared__ __align__(16) bf16 ztile[2][LC][ZS];
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

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kh = w >> 1, vh = w & 1;  // this wave's half of the rows, and of the columns
    const int D2 = p.D2, c0 = cb * LA_COLS;
    const int late = p.reverse ? 1 : 0;

    if (!STATES && a.s.cu && sg.p0 == 0 && (sg.n == 0 || sg.n == a.s.n_seqs - 1)) {
        // rows outside every sequence: zeros
        const int lo = sg.n == 0 ? 0 : a.s.T, hi = sg.n == 0 ? sg.t0 : a.s.T;
        for (int t = lo + (tid >> 2); t < hi; t += LA_THREADS / 4)
            *reinterpret_cast<u32x4*>(p.o + ((int64_t)t * H + h) * D2 + c0 + 8 * (tid & 3)) = u32x4{0, 0, 0, 0};
        if (sg.n == a.s.n_seqs - 1)
            for (int t = sg.t0 + sg.len + (tid >> 2); t < a.s.T; t += LA_THREADS / 4)
                *reinterpret_cast<u32x4*>(p.o + ((int64_t)t * H + h) * D2 + c0 + 8 * (tid & 3)) = u32x4{0, 0, 0, 0};
    }

    // ---- the state: accumulator element i of tile kt is row
    // channel(kh NT + kt, 4 g + i), column c0 + channel(vh, r)
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

    // ---- decays (natural logs; powers by exp2)
    const float ld = head_log_decay(a.log_decay, h);
    const float l2 = ld * LOG2E;
    const int i0 = 16 * w + r;  // this lane's query in the chunk
    float up = 0.f, dec[4][4], wz[2][8], c_s0, c_s1;
    if constexpr (!STATES) {
        up = exp2_hw((i0 + 1 - late) * l2) * p.x_scale;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) dec[d][i] = exp2_hw(max(16 * d + r - 4 * g - i, 0) * l2) * p.in_scale;
    }
    // weights of a chunk of n tokens, and its decay as c_s0 S + c_s1 S
    auto set_chunk = [&](int n) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int t = 32 * m + 16 * (e >> 2) + 4 * g + (e & 3);
                wz[m][e] = t < n ? exp2_hw((n - 1 - t + late) * l2) * p.z_scale : 0.f;
            }
        const float x = n * ld;
        const bool near = x > -0.6f;
        c_s0 = near ? 1.f : 0.f;
        c_s1 = near ? expm1f(x) : exp2_hw(n * l2);
    };

    // ---- rows of x, y, z at a position, and one position on
    const int64_t step = p.reverse ? -1 : 1;
    const int64_t tok0 = p.reverse ? (int64_t)sg.t0 + sg.len - 1 - sg.p0 : (int64_t)sg.t0 + sg.p0;
    const int64_t ystep = step * H * D1, zstep = step * H * D2;
    const uint16_t* const yrow = p.y + (tok0 * H + h) * D1;
    const uint16_t* const zrow = p.z + (tok0 * H + h) * D2 + c0;
    const uint16_t* const xrow = STATES ? nullptr : p.x + (tok0 * H + h) * D1;
    uint16_t* const orow = STATES ? nullptr : p.o + (tok0 * H + h) * D2 + c0;
    const int np = sg.p1 - sg.p0, nc = (np + LC - 1) / LC;

    u32x4 yreg[YV], zreg, xreg[KS];
    const u32x4 zero4 = {0, 0, 0, 0};
    auto load_yz = [&](int c) {
        const int n = np - c * LC;
#pragma unroll
        for (int i = 0; i < YV; ++i) {
            const int row = tid / TPR + i * (LA_THREADS / TPR);
            yreg[i] = row < n ? *reinterpret_cast<const u32x4*>(yrow + (int64_t)(c * LC + row) * ystep + 8 * (tid % TPR)) : zero4;
        }
        const int row = tid >> 2;
        zreg = row < n ? *reinterpret_cast<const u32x4*>(zrow + (int64_t)(c * LC + row) * zstep + 8 * (tid & 3)) : zero4;
    };
    auto load_x = [&](int c) {
        if constexpr (!STATES) {
            const int n = np - c * LC;
#pragma unroll
            for (int j = 0; j < KS; ++j)
                xreg[j] = i0 < n ? *reinterpret_cast<const u32x4*>(xrow + (int64_t)(c * LC + i0) * ystep + 32 * j + 8 * g) : zero4;
        }
    };
    auto put_yz = [&](int buf) {
#pragma unroll
        for (int i = 0; i < YV; ++i)
            *reinterpret_cast<u32x4*>(&ytile[buf][tid / TPR + i * (LA_THREADS / TPR)][8 * (tid % TPR)]) = yreg[i];
        *reinterpret_cast<u32x4*>(&ztile[buf][tid >> 2][8 * (tid & 3)]) = zreg;
    };
    auto put_s = [&](int buf) {
        if constexpr (!STATES) {
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                const bf16x8 f = join(to_bf16x4(S[2 * j]), to_bf16x4(S[2 * j + 1]));
                scopy[buf][vh][kh * (NT / 2) + j][lane] = __builtin_bit_cast(u32x4, f);
            }
        }
    };

    if (nc > 0) {
        set_chunk(min(np, LC));
        load_yz(0);
        load_x(0);
        put_yz(0);
        put_s(0);
        if (nc > 1) load_yz(1);
        __syncthreads();
    }
    for (int c = 0; c < nc; ++c) {
        const int buf = c & 1;
        const int n = min(np - c * LC, LC);
        bf16x8 xf[KS];
#pragma unroll
        for (int j = 0; j < KS; ++j) xf[j] = __builtin_bit_cast(bf16x8, xreg[j]);
        if (c + 1 < nc) {
            put_yz(buf ^ 1);
            load_x(c + 1);
        }
        if (c + 2 < nc) load_yz(c + 2);
        const bf16* yt = &ytile[buf][0][0];
        const bf16* zt = &ztile[buf][0][0];

        if constexpr (!STATES) {
            // S^T x: D rows are the columns channel(ct, .), D columns the queries
            floatx4 acc[2];
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                acc[ct] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < KS; ++j)
                    acc[ct] = mfma32(__builtin_bit_cast(bf16x8, scopy[buf][ct][j][lane]), xf[j], acc[ct]);
                acc[ct] *= up;
            }
            // P^T of the key tiles w, w - 1, ..., two at a time
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (2 * m <= w) {
                    bf16x4 pf[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int d = 2 * m + u;
                        floatx4 pt = {0.f, 0.f, 0.f, 0.f};
                        if (d <= w) {
#pragma unroll
                            for (int j = 0; j < KS; ++j)
                                pt = mfma32(*reinterpret_cast<const bf16x8*>(yt + (16 * (w - d) + r) * YS + 32 * j + 8 * g), xf[j], pt);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                pt[i] *= dec[d][i];
                                if (d == 0 && r < 4 * g + i) pt[i] = 0.f;
                            }
                        }
                        pf[u] = to_bf16x4(pt);
                    }
                    const int k0 = 16 * (w - 2 * m), k1 = max(k0 - 16, 0);
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct)
                        acc[ct] = mfma32(join(tile_t(zt + k0 * ZS, ZS, ct, lane), tile_t(zt + k1 * ZS, ZS, ct, lane)),
                                         join(pf[0], pf[1]), acc[ct]);
                }
            }
            if (i0 < n) {
                const bf16x8 ov = join(to_bf16x4(acc[0]), to_bf16x4(acc[1]));
                *reinterpret_cast<u32x4*>(orow + (int64_t)(c * LC + i0) * zstep + 8 * g) = __builtin_bit_cast(u32x4, ov);
            }
        }

        // ---- the state's update
        if (n < LC && c > 0) set_chunk(n);
#pragma unroll
        for (int kt = 0; kt < NT; ++kt)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[kt][i] = fmaf(S[kt][i], c_s1, S[kt][i] * c_s0);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const bf16x8 zf = join(tile_t(zt + 32 * m * ZS, ZS, vh, lane), tile_t(zt + (32 * m + 16) * ZS, ZS, vh, lane));
            bf16x8 z3[3];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = (float)zf[e] * wz[m][e];
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    z3[q][e] = (bf16)v;
                    v -= (float)z3[q][e];
                }
            }
#pragma unroll
            for (int kt = 0; kt < NT; ++kt) {
                const bf16x8 yf = join(tile_t(yt + 32 * m * YS, YS, kh * NT + kt, lane),
                                       tile_t(yt + (32 * m + 16) * YS, YS, kh * NT + kt, lane));
#pragma unroll
                for (int q = 2; q >= 0; --q) S[kt] = mfma32(yf, z3[q], S[kt]);
            }
        }
        if (c + 1 < nc) {
            put_s(buf ^ 1);
            __syncthreads();
        }
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
        if (states) hipLaunchKernelGGL((la_chunk_kernel<128, true>), grid, dim3(LA_THREADS), 0, stream, a);
        else hipLaunchKernelGGL((la_chunk_kernel<128, false>), grid, dim3(LA_THREADS), 0, stream, a);
    } else {
        if (states) hipLaunchKernelGGL((la_chunk_kernel<64, true>), grid, dim3(LA_THREADS), 0, stream, a);
        else hipLaunchKernelGGL((la_chunk_kernel<64, false>), grid, dim3(LA_THREADS), 0, stream, a);
    }
}

void launch_la_scan(const LaScanArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.s.n_seqs * a.s.H * (a.elems / 1024)), (unsigned)a.n_dirs);
    hipLaunchKernelGGL(la_scan_kernel, grid, dim3(256), 0, stream, a);
}

}  // namespace kda
