// la_api.hip -- the C ABI of linear attention with a decay for each head and
// of the gated norm (declared in include/kda.h): host-side argument checks,
// workspace layout and the launches on the caller's stream.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kda.h"
#include "la_launch.h"

namespace {

constexpr size_t ALIGN = 256;
constexpr int64_t I31 = (int64_t)1 << 31;
constexpr int32_t MAX_HEADS = 65536;  // 32-bit byte offsets within a chunk's rows

size_t align_up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool supported_dim(int32_t d) { return d == 64 || d == 128; }

struct LaCall {
    const int32_t* cu;
    bool packed;
    int32_t num_seqs, B, T, H, K, V;
    int32_t segments;  // the caller's request: chunks per segment, 0 automatic, < 0 whole
};

struct LaPlan {
    kda::LaSeqs s;
    bool narrow;  // whole sequences in workgroups of a few columns (la_narrow.hip)
};

// Kernel and segments (see LaSeqs) for `passes` passes over a batch side by side.
//
// A workgroup of la_chunk.hip has a (segment, head)'s whole rows, and a CU to itself:
// with fewer (sequence, head) pairs than CUs a sequence is cut into segments, which
// costs a second reading of y and z and two more launches: about 27 us and 4 us for
// every s chunks of 128 x 128, where s segments of every sequence are in flight.
// la_narrow.hip cuts the state's columns instead, which costs nothing but reads x and y
// once per 32 columns and z in 64-byte pieces: 1.25 us a chunk (0.85 with 64 rows), half
// as much again where more of its workgroups than CUs are in flight (512 are).  Forward
// (and backward) of H pairs, 128 x 128, in us, measured:
//             T = 1024     2048        4096          8192
//   H = 16    24 (25)     43 (44)     79 (80)       150 (153)   narrow
//             28 (51)     35 (54)     49 (78)        64 (127)   segments
//   H = 32    25 (37)     43 (64)     78 (120)      151 (270)   narrow
//             31 (56)     47 (89)     62 (126)       98 (222)   segments
//   H = 64    26          44          81            170         narrow
//             38 (53)     62 (89)     96 (169)      182 (338)   segments (backward: whole)
LaPlan plan(const LaCall& c, int passes) {
    LaPlan p{};
    kda::LaSeqs& s = p.s;
    s.cu = c.cu;
    s.n_seqs = c.packed ? c.num_seqs : c.B;
    s.T = c.T;
    s.H = c.H;
    s.seg_per_seq = 1;
    s.n_slots = s.n_seqs;
    const int64_t tokens = c.packed ? c.T : (int64_t)c.B * c.T;
    const int64_t chunks = (tokens / s.n_seqs + kda::LA_CHUNK - 1) / kda::LA_CHUNK;  // of an average sequence
    const int64_t pairs = (int64_t)s.n_seqs * c.H;
    const int64_t beside = pairs * passes;
    const int64_t most = std::max<int64_t>(1, chunks / 3);  // segments of three chunks or more
    const int64_t narrow_groups = kda::la_narrow_groups(pairs, std::max(c.K, c.V)) * passes;
    if (c.segments <= 0 && narrow_groups <= 512) {
        const double size = (c.K + c.V) / 256.0, s_flight = std::min<double>(256.0 / beside, (double)most);
        const bool rows64 = c.K == 64 && (passes == 1 || c.V == 64);
        const double narrow_us = chunks * (rows64 ? 0.85 : 1.25) * (narrow_groups > 256 ? 1.5 : 1.0);
        p.narrow = c.segments < 0 || narrow_us <= size * (27.0 + 4.0 * chunks / s_flight);
        if (p.narrow) return p;
    }
    int64_t per = c.segments;
    if (c.segments == 0) {
        per = -1;
        // one round of workgroups, or two where they leave fewer CUs idle
        int64_t n = 256 / beside;
        if (n >= 2 && 512 / beside > 2 * n) n = 512 / beside;
        n = std::min(n, most);
        if (n > 1) per = (chunks + n - 1) / n;
    }
    // (a segment that holds every token is the whole sequence)
    if (per > 0 && per * kda::LA_CHUNK < c.T) {
        s.seg_tokens = (int32_t)(per * kda::LA_CHUNK);
        if (c.packed) {
            const int64_t n = (int64_t)c.T / s.seg_tokens + s.n_seqs;
            s.n_slots = (int32_t)std::min<int64_t>(n, INT32_MAX);
        } else {
            s.seg_per_seq = (c.T + s.seg_tokens - 1) / s.seg_tokens;
            s.n_slots = (int32_t)std::min<int64_t>((int64_t)s.seg_per_seq * s.n_seqs, INT32_MAX);
        }
    } else if (c.packed && s.n_seqs <= 64 && beside > 256) {
        s.by_length = 1;
    }
    return p;
}

size_t la_states_bytes(const LaCall& c, const kda::LaSeqs& s) {
    return s.seg_tokens ? align_up((size_t)s.n_slots * c.H * c.K * c.V * sizeof(float)) : 0;
}

bool valid_sizes(const LaCall& c) {
    return c.B >= 1 && c.T >= 0 && c.H >= 1 && c.H <= MAX_HEADS && c.num_seqs >= 1 && supported_dim(c.K) && supported_dim(c.V) &&
           (int64_t)c.B * c.T < I31;
}

// Workgroups of a launch are counted in 32 bits: three passes over the slots and heads,
// sixteen pieces of a state.
bool countable(const kda::LaSeqs& s) { return (int64_t)s.n_slots * s.H < I31 / 64; }

// workspace bytes (dirs: 1 forward, 2 backward); 0: sizes that are not supported
size_t la_workspace(const LaCall& c, int dirs) {
    if (!valid_sizes(c)) return 0;
    const kda::LaSeqs s = plan(c, dirs == 2 ? 3 : 1).s;
    return countable(s) ? std::max(ALIGN, (size_t)dirs * la_states_bytes(c, s)) : 0;
}

// The same without knowing whether cu_seqlens will be passed: batches of these sizes plan
// alike but for the slots.  One row with num_seqs other than 1 is packed; else a B = 1
// batch may be either, and gets the larger of the two.
size_t la_any_workspace(int32_t B, int32_t T, int32_t H, int32_t K, int32_t V, int32_t num_seqs, int32_t segments,
                        int dirs) {
    const LaCall fixed{nullptr, false, num_seqs, B, T, H, K, V, segments};
    const size_t f = la_workspace(fixed, dirs);
    if (B != 1) return f;
    LaCall packed = fixed;
    packed.packed = true;
    const size_t p = la_workspace(packed, dirs);
    return num_seqs != 1 && !p ? 0 : std::max(f, p);
}

// Checks of every pass; fills the plan.
int check_la(const LaCall& c, float scale, const float* log_decay, const void* ws, size_t ws_bytes, int dirs,
             LaPlan& plan_out) {
    if (c.B < 1 || c.T < 0 || c.H < 1) return KDA_ERR_INVALID_ARG;
    if (!supported_dim(c.K) || !supported_dim(c.V)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)c.B * c.T >= I31 || !std::isfinite(scale) || !log_decay || !aligned(log_decay, 4))
        return KDA_ERR_INVALID_ARG;
    if (c.H > MAX_HEADS) return KDA_ERR_INVALID_ARG;
    if (c.packed && (c.B != 1 || c.num_seqs < 1 || !aligned(c.cu, 4))) return KDA_ERR_INVALID_ARG;
    plan_out = plan(c, dirs == 2 ? 3 : 1);
    const kda::LaSeqs& s = plan_out.s;
    if (!countable(s)) return KDA_ERR_INVALID_ARG;
    const size_t need = (size_t)dirs * la_states_bytes(c, s);
    if (need && (!ws || !aligned(ws, ALIGN) || ws_bytes < need)) return KDA_ERR_WORKSPACE;
    return KDA_OK;
}

kda::LaPass make_pass(const uint16_t* x, const uint16_t* y, const uint16_t* z, uint16_t* o, int32_t D1, int32_t D2,
                      int32_t row, int32_t col, bool reverse, float scale) {
    kda::LaPass p{};
    p.x = x;
    p.y = y;
    p.z = z;
    p.o = o;
    p.D1 = D1;
    p.D2 = D2;
    p.row = row;
    p.col = col;
    p.reverse = reverse;
    p.in_scale = scale;
    p.x_scale = reverse ? 1.f : scale;
    p.z_scale = reverse ? scale : 1.f;
    return p;
}

// what each segment adds to the state, for a pass with the states' own [K, V] layout
void launch_states(const kda::LaSeqs& s, const float* log_decay, const kda::LaPass* p, float* const* out, int n,
                   hipStream_t stream) {
    kda::LaArgs a{};
    a.s = s;
    a.log_decay = log_decay;
    for (int i = 0; i < n; ++i) {
        a.pass[i] = p[i];
        a.pass[i].x = nullptr;
        a.pass[i].o = nullptr;
        a.pass[i].s_in = nullptr;
        a.pass[i].s_out = out[i];
        a.pass[i].s_out_slots = 1;
    }
    kda::launch_la_chunk(a, n, true, stream);
}

void launch(const LaPlan& p, const kda::LaArgs& a, int n, hipStream_t stream) {
    if (p.narrow) kda::launch_la_narrow(a, n, stream);
    else kda::launch_la_chunk(a, n, false, stream);
}

int status() { return hipGetLastError() == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH; }

}  // namespace

extern "C" {

size_t la_fwd_workspace_size(int32_t B, int32_t T, int32_t H, int32_t K, int32_t V, int32_t num_seqs,
                             int32_t segment_chunks) {
    return la_any_workspace(B, T, H, K, V, num_seqs, segment_chunks, 1);
}

size_t la_bwd_workspace_size(int32_t B, int32_t T, int32_t H, int32_t K, int32_t V, int32_t num_seqs,
                             int32_t segment_chunks) {
    return la_any_workspace(B, T, H, K, V, num_seqs, segment_chunks, 2);
}

int la_fwd(const uint16_t* q, const uint16_t* k, const uint16_t* v, const float* log_decay, float scale,
           const float* initial_state, float* final_state, const int32_t* cu_seqlens, int32_t num_seqs, int32_t B,
           int32_t T, int32_t H, int32_t K, int32_t V, uint16_t* o, void* workspace, size_t workspace_bytes,
           int32_t segment_chunks, void* stream) {
    const LaCall c{cu_seqlens, cu_seqlens != nullptr, num_seqs, B, T, H, K, V, segment_chunks};
    LaPlan pl;
    const int st = check_la(c, scale, log_decay, workspace, workspace_bytes, 1, pl);
    if (st != KDA_OK) return st;
    const kda::LaSeqs& s = pl.s;
    if (T > 0 && (!q || !k || !v || !o)) return KDA_ERR_INVALID_ARG;
    for (const void* p : {(const void*)q, (const void*)k, (const void*)v, (const void*)o, (const void*)initial_state,
                          (const void*)final_state})
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const hipStream_t str = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();  // clear a stale error from unrelated work
    kda::LaArgs a{};
    a.s = s;
    a.log_decay = log_decay;
    kda::LaPass& p = a.pass[0];
    p = make_pass(q, k, v, o, K, V, V, 1, false, scale);
    p.s_in = initial_state;
    p.s_out = final_state;
    if (s.seg_tokens) {
        float* states = static_cast<float*>(workspace);
        launch_states(s, log_decay, &p, &states, 1, str);
        kda::LaScanArgs sc{};
        sc.s = s;
        sc.log_decay = log_decay;
        sc.init[0] = initial_state;
        sc.state[0] = states;
        sc.elems = K * V;
        sc.n_dirs = 1;
        kda::launch_la_scan(sc, str);
        p.s_in = states;
        p.s_in_slots = 1;
    }
    launch(pl, a, 1, str);
    return status();
}

int la_bwd(const uint16_t* q, const uint16_t* k, const uint16_t* v, const float* log_decay, float scale,
           const float* initial_state, const int32_t* cu_seqlens, int32_t num_seqs, int32_t B, int32_t T, int32_t H,
           int32_t K, int32_t V, const uint16_t* d_o, const float* d_final, uint16_t* dq, uint16_t* dk, uint16_t* dv,
           float* dh0, void* workspace, size_t workspace_bytes, int32_t segment_chunks, void* stream) {
    const LaCall c{cu_seqlens, cu_seqlens != nullptr, num_seqs, B, T, H, K, V, segment_chunks};
    LaPlan pl;
    const int st = check_la(c, scale, log_decay, workspace, workspace_bytes, 2, pl);
    if (st != KDA_OK) return st;
    const kda::LaSeqs& s = pl.s;
    if (T > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv)) return KDA_ERR_INVALID_ARG;
    for (const void* p : {(const void*)q, (const void*)k, (const void*)v, (const void*)d_o, (const void*)dq,
                          (const void*)dk, (const void*)dv, (const void*)initial_state, (const void*)d_final,
                          (const void*)dh0})
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const hipStream_t str = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    kda::LaPass pq = make_pass(d_o, v, k, dq, V, K, 1, V, false, scale);
    kda::LaPass pk = make_pass(v, d_o, q, dk, V, K, 1, V, true, scale);
    kda::LaPass pv = make_pass(k, q, d_o, dv, K, V, V, 1, true, scale);
    pq.s_in = initial_state;
    pk.s_in = pv.s_in = d_final;
    pv.s_out = dh0;
    if (s.seg_tokens) {
        float* states[2] = {static_cast<float*>(workspace),
                            static_cast<float*>(workspace) + la_states_bytes(c, s) / sizeof(float)};
        const kda::LaPass p[2] = {make_pass(q, k, v, nullptr, K, V, V, 1, false, scale), pv};
        launch_states(s, log_decay, p, states, 2, str);
        kda::LaScanArgs sc{};
        sc.s = s;
        sc.log_decay = log_decay;
        sc.init[0] = initial_state;
        sc.init[1] = d_final;
        sc.state[0] = states[0];
        sc.state[1] = states[1];
        sc.elems = K * V;
        sc.n_dirs = 2;
        kda::launch_la_scan(sc, str);
        pq.s_in = states[0];
        pk.s_in = pv.s_in = states[1];
        pq.s_in_slots = pk.s_in_slots = pv.s_in_slots = 1;
    }
    kda::LaArgs a{};
    a.s = s;
    a.log_decay = log_decay;
    a.pass[0] = pk;
    a.pass[1] = pv;
    a.pass[2] = pq;
    launch(pl, a, 3, str);
    return status();
}

int la_decode(const uint16_t* q, const uint16_t* k, const uint16_t* v, const float* log_decay, float scale,
              const float* state_in, float* state_out, int32_t N, int32_t H, int32_t K, int32_t V, uint16_t* o,
              void* stream) {
    if (N < 1 || H < 1) return KDA_ERR_INVALID_ARG;
    if (!q || !k || !v || !log_decay || !state_out || !o) return KDA_ERR_INVALID_ARG;
    if (!supported_dim(K) || !supported_dim(V)) return KDA_ERR_UNSUPPORTED;
    if (!std::isfinite(scale) || (int64_t)N * H * (V / 64) >= I31) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 8) || !aligned(o, 8) || !aligned(log_decay, 4) ||
        !aligned(state_in, 16) || !aligned(state_out, 16))
        return KDA_ERR_INVALID_ARG;
    kda::LaDecodeArgs d{};
    d.q = q;
    d.k = k;
    d.v = v;
    d.log_decay = log_decay;
    d.state_in = state_in;
    d.state_out = state_out;
    d.o = o;
    d.scale = scale;
    d.H = H;
    d.V = V;
    d.n_pairs = N * H;
    (void)hipGetLastError();
    kda::launch_la_decode(d, K, static_cast<hipStream_t>(stream));
    return status();
}

}  // extern "C"

namespace {

int check_norm(const uint16_t* x, const uint16_t* gate, const float* weight, const uint16_t* residual,
               const float* residual_scale, int32_t activation, float eps, int64_t tokens, int32_t H, int32_t D) {
    if (tokens < 0 || H < 1 || D < 1) return KDA_ERR_INVALID_ARG;
    if (D % 8 || D > 512) return KDA_ERR_UNSUPPORTED;
    if (tokens * (double)H >= (double)I31) return KDA_ERR_INVALID_ARG;
    if (activation != KDA_GATE_SIGMOID && activation != KDA_GATE_SILU) return KDA_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !weight) return KDA_ERR_INVALID_ARG;
    // (the scale says that there is a residual: it is never empty)
    if (residual && !residual_scale) return KDA_ERR_INVALID_ARG;
    if (tokens > 0 && (!x || (residual_scale && !residual))) return KDA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(gate, 16) || !aligned(residual, 16) || !aligned(weight, 4) ||
        !aligned(residual_scale, 4))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

kda::GatedNormArgs norm_args(const uint16_t* x, const uint16_t* gate, const float* weight, const uint16_t* residual,
                             const float* residual_scale, int32_t activation, float eps, int64_t tokens, int32_t H,
                             int32_t D) {
    kda::GatedNormArgs a{};
    a.x = x;
    a.gate = gate;
    a.weight = weight;
    a.res = residual;
    a.res_scale = residual_scale;
    a.silu = activation == KDA_GATE_SILU;
    a.eps = eps;
    a.H = H;
    a.D = D;
    a.rows = tokens * H;
    return a;
}

}  // namespace

extern "C" {

int gated_norm_fwd(const uint16_t* x, const uint16_t* gate, const float* weight, const uint16_t* residual,
                   const float* residual_scale, int32_t activation, float eps, int64_t tokens, int32_t H, int32_t D,
                   uint16_t* y, void* stream) {
    const int st = check_norm(x, gate, weight, residual, residual_scale, activation, eps, tokens, H, D);
    if (st != KDA_OK) return st;
    if (!aligned(y, 16) || (tokens > 0 && !y)) return KDA_ERR_INVALID_ARG;
    if (tokens == 0) return KDA_OK;
    kda::GatedNormArgs a = norm_args(x, gate, weight, residual, residual_scale, activation, eps, tokens, H, D);
    a.y = y;
    (void)hipGetLastError();
    kda::launch_gated_norm_fwd(a, static_cast<hipStream_t>(stream));
    return status();
}

size_t gated_norm_bwd_workspace_size(int64_t tokens, int32_t H, int32_t D) {
    if (tokens < 0 || H < 1 || D < 1 || D % 8 || D > 512 || tokens * (double)H >= (double)I31) return 0;
    const int64_t rows = tokens * H;
    return align_up((size_t)kda::gated_norm_groups(rows, D) * D * sizeof(float)) +
           align_up((size_t)rows * sizeof(float));
}

int gated_norm_bwd(const uint16_t* x, const uint16_t* gate, const float* weight, const uint16_t* residual,
                   const float* residual_scale, int32_t activation, float eps, int64_t tokens, int32_t H, int32_t D,
                   const uint16_t* dy, uint16_t* dx, uint16_t* dgate, float* dweight, uint16_t* dresidual,
                   float* dresidual_scale, void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_norm(x, gate, weight, residual, residual_scale, activation, eps, tokens, H, D);
    if (st != KDA_OK) return st;
    if (!dweight || (tokens > 0 && (!dy || !dx))) return KDA_ERR_INVALID_ARG;
    if ((gate && !dgate) || (residual && !dresidual) || (residual_scale && !dresidual_scale))
        return KDA_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(dx, 16) || !aligned(dgate, 16) || !aligned(dresidual, 16) ||
        !aligned(dweight, 4) || !aligned(dresidual_scale, 4))
        return KDA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, ALIGN) || workspace_bytes < gated_norm_bwd_workspace_size(tokens, H, D))
        return KDA_ERR_WORKSPACE;
    kda::GatedNormArgs a = norm_args(x, gate, weight, residual, residual_scale, activation, eps, tokens, H, D);
    a.dy = dy;
    a.dx = dx;
    a.dgate = dgate;
    a.dres = dresidual;
    a.dweight = dweight;
    a.dres_scale = dresidual_scale;
    a.groups = kda::gated_norm_groups(a.rows, D);
    a.part_w = static_cast<float*>(workspace);
    a.row_ds = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                        align_up((size_t)a.groups * D * sizeof(float)));
    (void)hipGetLastError();
    kda::launch_gated_norm_bwd(a, static_cast<hipStream_t>(stream));
    return status();
}

}  // extern "C"
