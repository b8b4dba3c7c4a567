// The launchers of the paged attention and the row sampler over a stand-in for
// the CUDA runtime with two devices (no GPU): each device has had a kernel's
// shared-memory attribute set before a launch that needs it, and grids follow
// the device's own number of SMs.  Links the library's object files.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <map>
#include <mutex>
#include <thread>
#include <vector>

#include "../../decoder_only_transformer_llama_b200/csrc/paged.h"

namespace {
thread_local int t_dev = 0;
thread_local dim3 t_grid, t_block;
thread_local size_t t_smem = 0;
thread_local cudaStream_t t_stream = nullptr;
std::mutex g_mu;
std::map<std::pair<int, const void*>, int> g_smem;      // (device, kernel) -> largest dynamic shared memory
int g_launches = 0, g_refused = 0, g_wide = 0;
constexpr int kSms[2] = {148, 20};
constexpr int kResident = 2;

cudaError_t launched(const void* f, dim3 grid, size_t smem) {
    std::lock_guard<std::mutex> lock(g_mu);
    ++g_launches;
    const auto it = g_smem.find({t_dev, f});
    const int most = it == g_smem.end() ? 48 * 1024 : it->second;
    if (smem > static_cast<size_t>(most)) { ++g_refused; return cudaErrorInvalidValue; }
    if (grid.x > static_cast<unsigned>(kSms[t_dev] * kResident)) ++g_wide;
    return cudaSuccess;
}
CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}
}  // namespace

extern "C" {
void** __cudaRegisterFatBinary(void*) { static void* h = nullptr; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t smem, cudaStream_t st) {
    t_grid = g; t_block = b; t_smem = smem; t_stream = st;
    return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* g, dim3* b, size_t* smem, void* st) {
    *g = t_grid; *b = t_block; *smem = t_smem; *static_cast<cudaStream_t*>(st) = t_stream;
    return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) { *d = t_dev; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int dev) { *v = kSms[dev]; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
    std::lock_guard<std::mutex> lock(g_mu);
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) g_smem[{t_dev, f}] = v;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
    *n = kResident;
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPoint(const char*, void** fn, unsigned long long, cudaDriverEntryPointQueryResult* q) {
    *fn = reinterpret_cast<void*>(&encode);
    if (q) *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernel(const void* f, dim3 grid, dim3, void**, size_t smem, cudaStream_t) { return launched(f, grid, smem); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
    return launched(f, dim3(1), c->dynamicSmemBytes);      // the sampler's grid follows its rows alone
}
}

namespace llb {
void set_error(const char*, ...) {}
void count_launch() {}
int cuda_fail(cudaError_t, const char*) { return LLAMA_ERR_CUDA; }
}  // namespace llb

int main() {
    alignas(256) static unsigned char mem[256];
    auto all = [&](int dev) {
        t_dev = dev;
        int bad = 0;
        for (int hd : {32, 64, 128})
            for (int dtype : {LLAMA_F32, LLAMA_BF16, LLAMA_F16})
                for (int B : {3, 200, 900})
                    for (int max_new : {1, 500}) {
                        llb::PagedAttnArgs a = {};
                        a.q = a.k_pages = a.v_pages = mem;
                        a.T = 4000; a.nh = 8; a.nkv = 2; a.hd = hd; a.B = B;
                        a.cu_new = a.seq_lens = a.block_tables = reinterpret_cast<const int32_t*>(mem);
                        a.max_pages = 100; a.n_pages = 1000; a.page_shift = 6; a.max_new = max_new; a.scale = 0.1f;
                        a.out = a.workspace = mem;
                        bad += llb::launch_paged_attention(a, dtype, nullptr) != LLAMA_OK;
                    }
        const float* f = reinterpret_cast<const float*>(mem);
        for (int B : {4, 50, 100})
            for (int V : {1000, 120000, 262144})
                bad += llb::launch_sample_rows(f, B, V, f, nullptr, f, f, f, reinterpret_cast<int32_t*>(mem), nullptr) != LLAMA_OK;
        return bad;
    };
    // the first calls on both devices come from several host threads at once
    int bad = 0;
    std::vector<std::thread> threads;
    for (int i = 0; i < 8; ++i)
        threads.emplace_back([&, i] {
            const int n = all(i % 2);
            std::lock_guard<std::mutex> lock(g_mu);
            bad += n;
        });
    for (auto& t : threads) t.join();
    for (int dev : {0, 1, 0}) bad += all(dev);
    printf("%d launches, %d refused, %d failed calls, %d grids past the device\n", g_launches, g_refused, bad, g_wide);
    if (bad || g_refused || g_wide || g_launches != 11 * (54 + 9)) return 1;
    printf("ok\n");
    return 0;
}
