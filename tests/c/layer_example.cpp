// layer_example.cpp -- layer norm, attention and AdamW through the C++ layer
// (include/basp.hpp) as a C++ caller uses them.  Test program.
//   layer_example        host-only: sizes and refusals, as exceptions
//   layer_example gpu    also small cases whose results are known
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include <cuda_runtime_api.h>

#include "basp.hpp"

#define CHECK(cond, msg)                                               \
    do {                                                               \
        if (!(cond)) {                                                 \
            std::fprintf(stderr, "layer_example: %s\n", msg);          \
            std::exit(1);                                              \
        }                                                              \
    } while (0)

template <typename F>
static basp_status refused(F f) {
    try {
        f();
    } catch (const basp::Error &e) {
        CHECK(std::strlen(e.what()) > 0, "a refusal says what is wrong");
        return e.status();
    }
    return BASP_OK;
}

static const basp_attention_desc kDesc = {1, 130, 130, 2, 1, 64, 40, 3, 0.125f, BASP_DTYPE_BF16};

static void host_checks() {
    CHECK(basp_layernorm_backward_workspace(100, 256) > 0, "workspace of the norm");
    CHECK(basp_attention_backward_workspace(&kDesc) > 0, "workspace of the attention");
    const basp_heads none = {nullptr, 0, 0, 0};
    CHECK(refused([&] { basp::attention(kDesc, none, none, none, none, nullptr, nullptr); }) == BASP_ERR_INVALID_ARG,
          "attention of nothing");
    CHECK(refused([&] { basp::attention_decode(kDesc, none, none, none, nullptr, none, nullptr, 0, nullptr); }) ==
              BASP_ERR_INVALID_ARG, "a token is one query");
    CHECK(refused([] {
              basp::layernorm(BASP_DTYPE_BF16, 4, 128, nullptr, 128, nullptr, 0, nullptr, nullptr, BASP_DTYPE_BF16,
                              1e-6f, nullptr, 0, nullptr, 0, nullptr, nullptr, nullptr, nullptr);
          }) == BASP_ERR_INVALID_ARG, "norm of nothing");
    basp_adamw_options o = {1e-3, 0.9, 0.999, 1e-8, 0.01, 0, nullptr, 0};
    CHECK(refused([&] { basp::adamw(nullptr, 0, o, nullptr); }) == BASP_ERR_INVALID_ARG, "steps count from 1");
    o.step = 1;
    CHECK(refused([&] { basp::adamw(nullptr, 0, o, nullptr); }) == BASP_OK, "a step over no tensors");
}

#define CUDA(x) CHECK((x) == cudaSuccess, #x)

struct Buffer {
    void *p = nullptr;
    explicit Buffer(size_t n) { CUDA(cudaMalloc(&p, n)); }
    ~Buffer() { cudaFree(p); }
    Buffer(const Buffer &) = delete;
    Buffer &operator=(const Buffer &) = delete;
    float *f() { return static_cast<float *>(p); }
};

static uint16_t bf16(float x) {                      // of values that it holds
    uint32_t u;
    std::memcpy(&u, &x, 4);
    return uint16_t(u >> 16);
}
static float from_bf16(uint16_t x) {
    const uint32_t u = uint32_t(x) << 16;
    float f;
    std::memcpy(&f, &u, 4);
    return f;
}

static void gpu_checks() {
    cudaStream_t stream;
    CUDA(cudaStreamCreate(&stream));

    // q = 0: every visible key weighs the same, and o is the mean of their values
    const int64_t S = kDesc.q_len, H = kDesc.q_heads, d = kDesc.head_dim;
    std::vector<uint16_t> v(S * d), out(S * H * d);
    for (int64_t j = 0; j < S; ++j)
        for (int64_t e = 0; e < d; ++e) v[j * d + e] = bf16(float((j * 7 + e * 3) % 32));
    Buffer q(S * H * d * 2), k(S * d * 2), vd(S * d * 2), o(S * H * d * 2), lse(S * H * 4);
    CUDA(cudaMemset(q.p, 0, S * H * d * 2));
    CUDA(cudaMemcpy(k.p, v.data(), S * d * 2, cudaMemcpyHostToDevice));
    CUDA(cudaMemcpy(vd.p, v.data(), S * d * 2, cudaMemcpyHostToDevice));
    const basp_heads hq = {q.p, S * H * d, H * d, d}, hk = {k.p, S * d, d, d}, hv = {vd.p, S * d, d, d};
    const basp_heads ho = {o.p, S * H * d, H * d, d};
    basp::attention(kDesc, hq, hk, hv, ho, lse.f(), stream);
    CUDA(cudaStreamSynchronize(stream));
    CUDA(cudaMemcpy(out.data(), o.p, S * H * d * 2, cudaMemcpyDeviceToHost));
    for (int64_t i = 0; i < S; ++i)
        for (int64_t e = 0; e < d; ++e) {
            double sum = 0;
            int n = 0;
            for (int64_t j = 0; j <= i; ++j)
                if (j > i - kDesc.window || j < kDesc.sinks) {
                    sum += (j * 7 + e * 3) % 32;
                    ++n;
                }
            // one rounding of the result (2^-8), 2^-20 for all else
            for (int64_t h = 0; h < H; ++h)
                CHECK(std::fabs(from_bf16(out[(i * H + h) * d + e]) - sum / n) <= (sum / n) * (1.0 / 256 + 1e-5),
                      "attention with equal weights");
        }

    // the same cache, one token, and the gradient of a constant's sum: dv sums to do's
    basp_attention_desc one = kDesc;
    one.q_len = 1;
    const int32_t len = int32_t(S);
    Buffer lengths(4), ws(size_t(basp_attention_decode_workspace(&one)) + 16), o1(H * d * 2);
    CUDA(cudaMemcpy(lengths.p, &len, 4, cudaMemcpyHostToDevice));
    const basp_heads h1 = {o1.p, H * d, H * d, d};
    basp::attention_decode(one, hq, hk, hv, static_cast<const int32_t *>(lengths.p), h1, ws.p,
                           size_t(basp_attention_decode_workspace(&one)), stream);
    CUDA(cudaStreamSynchronize(stream));
    std::vector<uint16_t> last(H * d);
    CUDA(cudaMemcpy(last.data(), o1.p, H * d * 2, cudaMemcpyDeviceToHost));
    for (int64_t e = 0; e < H * d; ++e)
        CHECK(std::fabs(from_bf16(last[e]) - from_bf16(out[(S - 1) * H * d + e])) <= from_bf16(last[e]) / 64, "one token");
    const int64_t bytes = basp_attention_backward_workspace(&kDesc);
    Buffer wb(bytes), g(S * H * d * 2), dq(S * H * d * 2), dk(S * d * 2), dv(S * d * 2);
    std::vector<uint16_t> ones(S * H * d, bf16(1.0f)), got(S * d);
    CUDA(cudaMemcpy(g.p, ones.data(), S * H * d * 2, cudaMemcpyHostToDevice));
    basp::attention_backward(kDesc, hq, hk, hv, ho, lse.f(), {g.p, S * H * d, H * d, d}, {dq.p, S * H * d, H * d, d},
                             {dk.p, S * d, d, d}, {dv.p, S * d, d, d}, wb.p, size_t(bytes), stream);
    CUDA(cudaStreamSynchronize(stream));
    CUDA(cudaMemcpy(got.data(), dv.p, S * d * 2, cudaMemcpyDeviceToHost));
    double sum = 0;
    for (uint16_t x : got) sum += from_bf16(x);
    CHECK(std::fabs(sum / (S * H * d) - 1) <= 1.0 / 128, "every query's weights sum to 1");
    unsigned long long timeouts = 1;
    CHECK(basp_attention_timeouts(&timeouts) == BASP_OK && timeouts == 0, "no wait ran out");

    // rows of 1, -1, 1, -1, ...: mean 0, variance 1
    const int64_t M = 3, N = 256;
    std::vector<float> x(M * N), w(N, 2.0f), b(N, 0.5f), y(M * N);
    for (int64_t i = 0; i < M * N; ++i) x[i] = i % 2 ? -1.0f : 1.0f;
    Buffer xd(M * N * 4), wd(N * 4), bd(N * 4), yd(M * N * 4);
    CUDA(cudaMemcpy(xd.p, x.data(), M * N * 4, cudaMemcpyHostToDevice));
    CUDA(cudaMemcpy(wd.p, w.data(), N * 4, cudaMemcpyHostToDevice));
    CUDA(cudaMemcpy(bd.p, b.data(), N * 4, cudaMemcpyHostToDevice));
    basp::layernorm(BASP_DTYPE_FP32, M, N, xd.p, N, nullptr, 0, wd.p, bd.p, BASP_DTYPE_FP32, 0.0f, nullptr, 0, yd.p, N,
                    nullptr, nullptr, nullptr, stream);
    // the first step of Adam is lr times the gradient's sign
    std::vector<float> p(N, 1.0f), grad(N);
    for (int64_t i = 0; i < N; ++i) grad[i] = i % 3 ? 0.25f : -4.0f;
    Buffer pd(N * 4), gd(N * 4), m1(N * 4), v1(N * 4);
    CUDA(cudaMemcpy(pd.p, p.data(), N * 4, cudaMemcpyHostToDevice));
    CUDA(cudaMemcpy(gd.p, grad.data(), N * 4, cudaMemcpyHostToDevice));
    CUDA(cudaMemset(m1.p, 0, N * 4));
    CUDA(cudaMemset(v1.p, 0, N * 4));
    const basp_adamw_tensor t = {pd.p, gd.p, m1.p, v1.p, nullptr, nullptr, N, BASP_DTYPE_FP32, BASP_DTYPE_FP32};
    basp::adamw(&t, 1, {0.125, 0.9, 0.999, 0, 0, 1, nullptr, 0}, stream);
    CUDA(cudaStreamSynchronize(stream));
    CUDA(cudaMemcpy(y.data(), yd.p, M * N * 4, cudaMemcpyDeviceToHost));
    CUDA(cudaMemcpy(p.data(), pd.p, N * 4, cudaMemcpyDeviceToHost));
    for (int64_t i = 0; i < M * N; ++i) CHECK(std::fabs(y[i] - (i % 2 ? -1.5f : 2.5f)) <= 1e-6f, "norm");
    for (int64_t i = 0; i < N; ++i) CHECK(std::fabs(p[i] - (i % 3 ? 0.875f : 1.125f)) <= 1e-6f, "first step");
    CUDA(cudaStreamDestroy(stream));
}

int main(int argc, char **argv) {
    host_checks();
    if (argc > 1 && std::strcmp(argv[1], "gpu") == 0) gpu_checks();
    std::puts("layer_example ok");
    return 0;
}
