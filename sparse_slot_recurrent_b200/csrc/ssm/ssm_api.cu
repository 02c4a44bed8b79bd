// ssm_api.cu -- the C ABI of the state space layer's operators: argument checks and launches.
// Nothing here allocates device memory.
#include <cstdarg>
#include <cstdio>

#include "../../../include/ramnet.h"
#include "ssm.h"

namespace ramnet {
ramnet_status set_last_error(ramnet_status s, const char* msg);  // ramnet_api.cu
}

namespace {

ramnet_status fail(ramnet_status s, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return ramnet::set_last_error(s, buf);
}

ramnet_status launched(cudaError_t e, const char* what)
{
    if (e != cudaSuccess) return fail(RAMNET_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return RAMNET_OK;
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_dtype(ramnet_dtype d) { return d == RAMNET_F32 || d == RAMNET_BF16; }
size_t elem(ramnet_dtype d) { return d == RAMNET_BF16 ? 2 : 4; }

// The status word for kernels that only record failed range checks, of the build that makes these.
uint32_t* check_word()
{
#ifdef RAMNET_DEBUG
    return ramnet::library_status_word();
#else
    return nullptr;
#endif
}

#define CHECK(cond, ...)                                            \
    do {                                                            \
        if (!(cond)) return fail(RAMNET_ERR_INVALID_ARG, __VA_ARGS__); \
    } while (0)
#define NEED(p, n)                                                  \
    do {                                                            \
        CHECK((p) != nullptr, "%s is NULL", #p);                    \
        CHECK(aligned(p, n), "%s not %zu-byte aligned", #p, (size_t)(n)); \
    } while (0)
#define MAY(p, n) CHECK((p) == nullptr || aligned(p, n), "%s not %zu-byte aligned", #p, (size_t)(n))

// Longest sequence or row, and most channels of a token of the scan: indices may run a block past the end without leaving
// 32 bits.
constexpr int64_t kLongest = 1ll << 30;

bool side(int32_t n) { return n == 16 || n == 32 || n == 64 || n == 128 || n == 256; }

ramnet_status check_ssm(const ramnet_ssm_config* c, int64_t B, int64_t T)
{
    CHECK(c != nullptr, "cfg is NULL");
    CHECK(side(c->N), "N=%d not in {16,32,64,128,256}", c->N);
    CHECK(side(c->P), "P=%d not in {16,32,64,128,256}", c->P);
    CHECK(c->H >= 1 && c->G >= 1 && c->H % c->G == 0, "G=%d does not divide H=%d", c->G, c->H);
    CHECK(c->dt_min <= c->dt_max, "dt_min and dt_max must be ordered numbers");
    CHECK(B >= 1 && T >= 1, "B and T must be >= 1");
    // (B*H first: the product of all three could pass 64 bits)
    CHECK(B * c->H <= (1ll << 27) - 1 && B * c->H * T <= (1ll << 31) - 1, "B*T*H too large");
    CHECK(T <= kLongest, "T too large");
    return RAMNET_OK;
}

ramnet_status check_prompt(const ramnet_ssm_config* c, int64_t B, int64_t T)
{
    const ramnet_status st = check_ssm(c, B, T);
    if (st != RAMNET_OK) return st;
    CHECK(static_cast<int64_t>(c->H) * c->P <= kLongest, "H*P too large");
    return RAMNET_OK;
}

// Strides of a [B,T,H,.] operand, dense if none are given; false if unusable.
bool take_strides(const ramnet_strides* s, int64_t B, int64_t T, int64_t H, int64_t last, ramnet::Str3* out)
{
    if (s == nullptr) {
        *out = {T * H * last, H * last, last};
        return true;
    }
    if (s->b < 0 || s->t < 0 || s->h < 0) return false;
    const double span = static_cast<double>(B - 1) * s->b + static_cast<double>(T - 1) * s->t +
                        static_cast<double>(H - 1) * s->h + static_cast<double>(last);
    *out = {s->b, s->t, s->h};
    return span <= 2.0e18;
}

size_t state_bytes(const ramnet_ssm_config* c, int64_t B) { return sizeof(float) * B * c->H * c->N * c->P; }

// The workspace: step sizes and decays by chunk of 64 tokens, then, where sequences are cut, the pieces' states
// and their decays; room for either form's cut.
struct Workspace {
    size_t state_off, decay_off, total;
};

Workspace ssm_workspace(const ramnet_ssm_config* c, int64_t B, int64_t T)
{
    Workspace w;
    const size_t heads = static_cast<size_t>(B) * c->H;
    size_t slots = 0;
    for (const ramnet::SsmSplit& s : {ramnet::ssm_split(B, T, c->H, c->G, c->P), ramnet::ssm_split_plain(B, T, c->H, c->N, c->P)})
        if (s.nseg > 1 && static_cast<size_t>(s.slots()) > slots) slots = s.slots();
    w.state_off = heads * ((T + ramnet::kChunk - 1) / ramnet::kChunk) * sizeof(ramnet::ChunkTok);
    w.decay_off = w.state_off + state_bytes(c, B) * slots;
    w.total = w.decay_off + sizeof(float) * heads * slots;
    return w;
}

}  // namespace

extern "C" {

size_t ramnet_ssm_workspace_bytes(const ramnet_ssm_config* cfg, int32_t B, int32_t T)
{
    ramnet::set_last_error(RAMNET_OK, "");
    if (check_prompt(cfg, B, T) != RAMNET_OK) return 0;
    return ssm_workspace(cfg, B, T).total;
}

ramnet_status ramnet_ssm_forward(const ramnet_ssm_config* cfg, int32_t B, int32_t T, ramnet_dtype in_dt, const void* x,
                                 const ramnet_strides* xs, const void* dt, const ramnet_strides* dts, const float* A,
                                 const void* Bm, const ramnet_strides* bs, const void* Cm, const ramnet_strides* cs,
                                 const float* D, const float* dt_bias, const int32_t* lengths, const float* S_in,
                                 void* y, ramnet_dtype out_dt, float* S_out, void* workspace, size_t workspace_bytes,
                                 void* stream)
{
    ramnet::set_last_error(RAMNET_OK, "");
    const ramnet_status st = check_prompt(cfg, B, T);
    if (st != RAMNET_OK) return st;
    CHECK(valid_dtype(in_dt) && valid_dtype(out_dt), "bad dtype");
    ramnet::SsmParams p{};
    CHECK(take_strides(xs, B, T, cfg->H, cfg->P, &p.xs), "bad strides of x");
    CHECK(take_strides(dts, B, T, cfg->H, 1, &p.dts), "bad strides of dt");
    CHECK(take_strides(bs, B, T, cfg->G, cfg->N, &p.bs), "bad strides of Bm");
    CHECK(take_strides(cs, B, T, cfg->G, cfg->N, &p.cs), "bad strides of Cm");
    const size_t es = elem(in_dt);
    NEED(x, es);
    NEED(dt, es);
    NEED(Bm, es);
    NEED(Cm, es);
    NEED(A, 4);
    MAY(D, 4);
    MAY(dt_bias, 4);
    MAY(lengths, 4);
    MAY(S_in, 16);
    NEED(y, 16);
    NEED(S_out, 16);
    const Workspace ws = ssm_workspace(cfg, B, T);
    NEED(workspace, 16);
    CHECK(workspace_bytes >= ws.total, "workspace of %zu bytes, %zu needed", workspace_bytes, ws.total);
    unsigned char* base = static_cast<unsigned char*>(workspace);
    p.toks = reinterpret_cast<ramnet::ChunkTok*>(base);
    p.seg_state = reinterpret_cast<float*>(base + ws.state_off);
    p.seg_decay = reinterpret_cast<float*>(base + ws.decay_off);
    p.x = x, p.dt = dt, p.A = A, p.Bm = Bm, p.Cm = Cm, p.D = D, p.dt_bias = dt_bias;
    p.in_bf16 = in_dt == RAMNET_BF16, p.out_bf16 = out_dt == RAMNET_BF16;
    p.lengths = lengths, p.S_in = S_in, p.y = y, p.S_out = S_out;
    p.B = B, p.T = T, p.H = cfg->H, p.G = cfg->G, p.N = cfg->N, p.P = cfg->P;
    p.softplus = cfg->dt_softplus != 0, p.dt_min = cfg->dt_min, p.dt_max = cfg->dt_max;
    const int polls = ramnet::scan_wait_ns() / ramnet::kPollNs;  // of one wait
    p.poll_cost = polls > 0 ? ramnet::kWaitNs / polls : ramnet::kWaitNs + 1;
    p.status = ramnet::library_status_word();
    if (p.status == nullptr) return launched(cudaGetLastError(), "status word");
    return launched(ramnet::launch_ssm_scan(p, static_cast<cudaStream_t>(stream)), "ssm_forward launch");
}

ramnet_status ramnet_ssm_step(const ramnet_ssm_config* cfg, int32_t B, ramnet_dtype in_dt, const void* x,
                              const ramnet_strides* xs, const void* dt, const ramnet_strides* dts, const float* A,
                              const void* Bm, const ramnet_strides* bs, const void* Cm, const ramnet_strides* cs,
                              const float* D, const float* dt_bias, float* S, void* y, ramnet_dtype out_dt,
                              void* stream)
{
    ramnet::set_last_error(RAMNET_OK, "");
    const ramnet_status st = check_ssm(cfg, B, 1);
    if (st != RAMNET_OK) return st;
    CHECK(valid_dtype(in_dt) && valid_dtype(out_dt), "bad dtype");
    ramnet::SsmStepParams p{};
    CHECK(take_strides(xs, B, 1, cfg->H, cfg->P, &p.xs), "bad strides of x");
    CHECK(take_strides(dts, B, 1, cfg->H, 1, &p.dts), "bad strides of dt");
    CHECK(take_strides(bs, B, 1, cfg->G, cfg->N, &p.bs), "bad strides of Bm");
    CHECK(take_strides(cs, B, 1, cfg->G, cfg->N, &p.cs), "bad strides of Cm");
    const size_t es = elem(in_dt);
    NEED(x, es);
    NEED(dt, es);
    NEED(Bm, es);
    NEED(Cm, es);
    NEED(A, 4);
    MAY(D, 4);
    MAY(dt_bias, 4);
    NEED(S, 16);
    NEED(y, 16);
    p.x = x, p.dt = dt, p.A = A, p.Bm = Bm, p.Cm = Cm, p.D = D, p.dt_bias = dt_bias;
    p.in_bf16 = in_dt == RAMNET_BF16, p.out_bf16 = out_dt == RAMNET_BF16;
    p.S = S, p.y = y, p.status = check_word();
    p.B = B, p.H = cfg->H, p.G = cfg->G, p.N = cfg->N, p.P = cfg->P;
    p.softplus = cfg->dt_softplus != 0, p.dt_min = cfg->dt_min, p.dt_max = cfg->dt_max;
    return launched(ramnet::launch_ssm_step(p, static_cast<cudaStream_t>(stream)), "ssm_step launch");
}

ramnet_status ramnet_conv_forward(int32_t B, int32_t T, int32_t C, int32_t W, ramnet_dtype in_dt, const void* x,
                                  int64_t x_b, int64_t x_t, const float* w, const float* bias, int32_t silu,
                                  const int32_t* lengths, const void* state_in, void* y, ramnet_dtype out_dt,
                                  void* state_out, void* stream)
{
    ramnet::set_last_error(RAMNET_OK, "");
    CHECK(B >= 1 && T >= 1 && C >= 1, "B, T, C must be >= 1");
    CHECK(static_cast<int64_t>(B) * T <= (1ll << 31) - 1 &&
              static_cast<int64_t>(B) * C <= (1ll << 31) - 1 &&
              static_cast<double>(B) * C * ((static_cast<int64_t>(T) + 15) / 16) <= 1.0e11,
          "B*T*C too large");
    CHECK(T <= kLongest, "T too large");
    CHECK(W >= 2 && W <= 4, "W=%d outside [2,4]", W);
    CHECK(valid_dtype(in_dt) && valid_dtype(out_dt), "bad dtype");
    ramnet::Str3 xs;
    const ramnet_strides given = {x_b, x_t, 0};
    CHECK(take_strides(&given, B, T, 1, C, &xs), "bad strides of x");
    const size_t es = elem(in_dt);
    NEED(x, es);
    NEED(w, 4);
    MAY(bias, 4);
    MAY(lengths, 4);
    MAY(state_in, 16);
    MAY(state_out, 16);
    NEED(y, 16);
    ramnet::ConvParams p{x, x_b, x_t, in_dt == RAMNET_BF16, w, bias, silu != 0, lengths, state_in, y,
                         out_dt == RAMNET_BF16, state_out, B, T, C, W, check_word()};
    return launched(ramnet::launch_conv(p, static_cast<cudaStream_t>(stream)), "conv_forward launch");
}

ramnet_status ramnet_conv_step(int32_t B, int32_t C, int32_t W, ramnet_dtype in_dt, const void* x, int64_t x_b,
                               const float* w, const float* bias, int32_t silu, void* state, void* y,
                               ramnet_dtype out_dt, void* stream)
{
    ramnet::set_last_error(RAMNET_OK, "");
    CHECK(B >= 1 && C >= 1, "B and C must be >= 1");
    CHECK(static_cast<int64_t>(B) * C <= (1ll << 31) - 1, "B*C too large");
    CHECK(W >= 2 && W <= 4, "W=%d outside [2,4]", W);
    CHECK(valid_dtype(in_dt) && valid_dtype(out_dt), "bad dtype");
    ramnet::Str3 xs;
    const ramnet_strides given = {x_b, 0, 0};
    CHECK(take_strides(&given, B, 1, 1, C, &xs), "bad stride of x");
    const size_t es = elem(in_dt);
    NEED(x, es);
    NEED(w, 4);
    MAY(bias, 4);
    NEED(state, 16);
    NEED(y, 16);
    ramnet::ConvStepParams p{x, x_b, in_dt == RAMNET_BF16, w, bias, silu != 0, state, y, out_dt == RAMNET_BF16, B, C, W, check_word()};
    return launched(ramnet::launch_conv_step(p, static_cast<cudaStream_t>(stream)), "conv_step launch");
}

ramnet_status ramnet_norm_gate(int64_t R, int32_t D, int32_t groups, ramnet_dtype in_dt, const void* x, int64_t x_r,
                               const void* z, int64_t z_r, const float* w, float eps, int32_t gate_first, void* y,
                               ramnet_dtype out_dt, void* stream)
{
    ramnet::set_last_error(RAMNET_OK, "");
    CHECK(R >= 1 && D >= 1, "R and D must be >= 1");
    CHECK(D <= kLongest, "D too large");
    CHECK(groups >= 1 && D % groups == 0, "groups=%d does not divide D=%d", groups, D);
    CHECK(R <= ((1ll << 31) - 1) / groups, "R*groups too large");
    CHECK(valid_dtype(in_dt) && valid_dtype(out_dt), "bad dtype");
    CHECK(eps >= 0.0f, "eps must be >= 0");
    ramnet::Str3 unused;
    const ramnet_strides xs = {x_r, 0, 0}, zs = {z_r, 0, 0};
    CHECK(take_strides(&xs, R, 1, 1, D, &unused), "bad row stride of x");
    CHECK(z == nullptr || take_strides(&zs, R, 1, 1, D, &unused), "bad row stride of z");
    const size_t es = elem(in_dt);
    NEED(x, es);
    MAY(z, es);
    MAY(w, 16);
    NEED(y, 16);
    ramnet::NormParams p{x, x_r, z, z_r, in_dt == RAMNET_BF16, w, y, out_dt == RAMNET_BF16, R, D, groups, eps, gate_first != 0, check_word()};
    return launched(ramnet::launch_norm_gate(p, static_cast<cudaStream_t>(stream)), "norm_gate launch");
}

}  // extern "C"
