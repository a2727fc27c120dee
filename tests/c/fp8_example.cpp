// fp8_example.cpp -- the 8-bit projections through the C++ layer
// (include/basp.hpp) as a C++ caller uses them.  Test program.
//   fp8_example        host-only: sizes and refusals, as exceptions
//   fp8_example gpu    also norm -> product and quantise -> product of small
//                      whole numbers, whose results are exact
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
            std::fprintf(stderr, "fp8_example: %s\n", msg);            \
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

static void host_checks() {
    CHECK(basp_rmsnorm_backward_workspace(100, 256) > 0, "workspace");
    CHECK(refused([] {
              basp::rmsnorm(BASP_DTYPE_BF16, 4, 128, nullptr, 128, nullptr, 0, nullptr, BASP_DTYPE_BF16, 1e-6f, nullptr,
                            0, nullptr, 0, nullptr, nullptr, nullptr);
          }) == BASP_ERR_INVALID_ARG, "norm of nothing");
    CHECK(refused([] {
              basp::quantize_fp8(BASP_DTYPE_BF16, 4, 128, nullptr, 128, nullptr, nullptr, nullptr);
          }) != BASP_OK, "quantiser without an output");
    CHECK(refused([] {
              basp_fp8_matrix a{nullptr, nullptr, 4, 128, 128, 4, 1}, b{nullptr, nullptr, 4, 256, 256, 4, 1};
              basp::matmul_fp8(a, b, nullptr, false, BASP_DTYPE_FP32, nullptr, 4, nullptr);
          }) != BASP_OK, "product of unequal lengths");
}

#define CUDA(x) CHECK((x) == cudaSuccess, #x)

struct Buffer {
    void *p = nullptr;
    explicit Buffer(size_t n) { CUDA(cudaMalloc(&p, n)); }
    ~Buffer() { cudaFree(p); }
    Buffer(const Buffer &) = delete;
    Buffer &operator=(const Buffer &) = delete;
};

static void gpu_checks() {
    const int64_t M = 5, N = 40, K = 256;
    std::vector<float> x(M * K), w(N * K), ones(K, 1.0f), c(M * N);
    for (int64_t i = 0; i < M * K; ++i) x[i] = float(i * 7 % 9) - 4;
    for (int64_t i = 0; i < N * K; ++i) w[i] = float(i * 5 % 7) - 3;
    Buffer dx(M * K * 4), dw(N * K * 4), dn(K * 4), dc(M * N * 4);
    Buffer xv(M * K), xs(M * 4), wv(N * K), ws(4);
    basp_fp8_matrix xq{xv.p, xs.p, M, K, K, 4, 1}, wq{wv.p, ws.p, N, K, K, 4, 128};
    cudaStream_t stream;
    CUDA(cudaStreamCreate(&stream));
    CUDA(cudaMemcpy(dx.p, x.data(), M * K * 4, cudaMemcpyHostToDevice));
    CUDA(cudaMemcpy(dw.p, w.data(), N * K * 4, cudaMemcpyHostToDevice));
    CUDA(cudaMemcpy(dn.p, ones.data(), K * 4, cudaMemcpyHostToDevice));
    basp::quantize_fp8(BASP_DTYPE_FP32, N, K, dw.p, K, &wq, nullptr, stream);
    basp::quantize_fp8(BASP_DTYPE_FP32, M, K, dx.p, K, &xq, nullptr, stream);
    basp::matmul_fp8(xq, wq, nullptr, false, BASP_DTYPE_FP32, dc.p, N, stream);
    basp::matmul_fp8(xq, wq, nullptr, true, BASP_DTYPE_FP32, dc.p, N, stream);
    CUDA(cudaStreamSynchronize(stream));
    CUDA(cudaMemcpy(c.data(), dc.p, M * N * 4, cudaMemcpyDeviceToHost));
    for (int64_t m = 0; m < M; ++m)
        for (int64_t n = 0; n < N; ++n) {
            float s = 0;
            for (int64_t k = 0; k < K; ++k) s += x[m * K + k] * w[n * K + k];
            CHECK(c[m * N + n] == 2 * s, "product of whole numbers");
        }
    // rows of +-2 have the root mean square 2: the norm gives +-1
    for (int64_t i = 0; i < M * K; ++i) x[i] = i % 3 ? 2.0f : -2.0f;
    CUDA(cudaMemcpy(dx.p, x.data(), M * K * 4, cudaMemcpyHostToDevice));
    basp::rmsnorm(BASP_DTYPE_FP32, M, K, dx.p, K, nullptr, 0, dn.p, BASP_DTYPE_FP32, 0.0f, nullptr, 0, nullptr, 0, &xq,
                  nullptr, stream);
    basp::matmul_fp8(xq, wq, nullptr, false, BASP_DTYPE_FP32, dc.p, N, stream);
    CUDA(cudaStreamSynchronize(stream));
    CUDA(cudaMemcpy(c.data(), dc.p, M * N * 4, cudaMemcpyDeviceToHost));
    for (int64_t m = 0; m < M; ++m)
        for (int64_t n = 0; n < N; ++n) {
            float s = 0;
            for (int64_t k = 0; k < K; ++k) s += x[m * K + k] / 2 * w[n * K + k];
            CHECK(c[m * N + n] == s, "norm and product");
        }
    unsigned long long count = 1;
    CHECK(basp_matmul_fp8_timeouts(&count) == BASP_OK && count == 0, "no wait ran out");
    CUDA(cudaStreamDestroy(stream));
}

int main(int argc, char **argv) {
    host_checks();
    if (argc > 1 && std::strcmp(argv[1], "gpu") == 0) gpu_checks();
    std::printf("fp8_example ok\n");
    return 0;
}
