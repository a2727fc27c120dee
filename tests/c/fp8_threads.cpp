// fp8_threads.cpp -- the norm from several host threads at once, through the C++
// layer (include/basp.hpp): each thread has a stream of its own and rows of its
// own length.  Test program (needs a GPU): exit status 0 and "fp8_threads ok".
#include <atomic>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>

#include <cuda_runtime_api.h>

#include "basp.hpp"

#define CHECK(cond, msg)                                               \
    do {                                                               \
        if (!(cond)) {                                                 \
            std::fprintf(stderr, "fp8_threads: %s\n", msg);            \
            std::exit(1);                                              \
        }                                                              \
    } while (0)
#define CUDA(x) CHECK((x) == cudaSuccess, #x)

namespace {

// many rows: the kernels whose shared memory follows the number of columns
constexpr int64_t kRows = 400;
constexpr int kCalls = 5000;

float *device_floats(size_t n) {
    void *p = nullptr;
    CUDA(cudaMalloc(&p, n * sizeof(float)));
    return static_cast<float *>(p);
}

// Norms of one shape forward and backward.  Rows of +-2 have the root mean
// square 2: the norm gives +-1, and its own output as the gradient gives zero.
struct Caller {
    int64_t cols;
    float *x = nullptr, *w = nullptr, *y = nullptr, *dx = nullptr, *rstd = nullptr;
    cudaStream_t stream = nullptr;

    explicit Caller(int64_t n) : cols(n) {
        std::vector<float> hx(size_t(kRows * cols)), ones(size_t(cols), 1.0f);
        for (size_t i = 0; i < hx.size(); ++i) hx[i] = i % 3 ? 2.0f : -2.0f;
        x = device_floats(hx.size());
        y = device_floats(hx.size());
        dx = device_floats(hx.size());
        w = device_floats(ones.size());
        rstd = device_floats(kRows);
        CUDA(cudaMemcpy(x, hx.data(), hx.size() * 4, cudaMemcpyHostToDevice));
        CUDA(cudaMemcpy(w, ones.data(), size_t(cols) * 4, cudaMemcpyHostToDevice));
        CUDA(cudaStreamCreate(&stream));
    }
    void run(std::atomic<int> &errors) {
        for (int i = 0; i < kCalls; ++i) {
            try {
                basp::rmsnorm(BASP_DTYPE_FP32, kRows, cols, x, cols, nullptr, 0, w, BASP_DTYPE_FP32, 0.0f, nullptr, 0,
                              y, cols, nullptr, rstd, stream);
                basp::rmsnorm_backward(BASP_DTYPE_FP32, kRows, cols, y, cols, x, cols, rstd, w, BASP_DTYPE_FP32,
                                       nullptr, 0, dx, cols, nullptr, nullptr, 0, stream);
            } catch (const basp::Error &) {
                ++errors;
            }
        }
    }
    void check() {
        std::vector<float> hy(size_t(kRows * cols)), hd(hy.size());
        CUDA(cudaStreamSynchronize(stream));
        CUDA(cudaMemcpy(hy.data(), y, hy.size() * 4, cudaMemcpyDeviceToHost));
        CUDA(cudaMemcpy(hd.data(), dx, hd.size() * 4, cudaMemcpyDeviceToHost));
        for (size_t i = 0; i < hy.size(); ++i)
            CHECK(hy[i] == (i % 3 ? 1.0f : -1.0f) && hd[i] > -1e-5f && hd[i] < 1e-5f, "values of a thread's norm");
    }
};

}  // namespace

int main() {
    Caller callers[] = {Caller(2048), Caller(768), Caller(1536), Caller(1024)};
    std::atomic<int> errors{0};
    std::vector<std::thread> threads;
    for (Caller &c : callers) threads.emplace_back([&c, &errors] { c.run(errors); });
    for (std::thread &t : threads) t.join();
    if (errors != 0) {
        std::fprintf(stderr, "fp8_threads: %d calls of %d failed\n", errors.load(), 4 * kCalls);
        return 1;
    }
    for (Caller &c : callers) c.check();
    std::printf("fp8_threads ok\n");
    return 0;
}
