// Copies of a product's operands with their rows on 16 bytes (prod_api.hpp).
#include "prod_api.hpp"

namespace tg {

struct CopyArgs {
    const char *src[3];
    char *dst[3];
    int64_t lds[3], first[4];                          // bytes; chunks before an operand
    int64_t ldd;
    int kbytes, chunks;                                // of a row
};

// A chunk of 16 bytes a thread: the row's last one with zeros past its end.
// Bound by memory (12286 rows of 2002 bytes 11.4 us, 4.6 TB/s with both).
template <int T>
__global__ void __launch_bounds__(256) prod_copy_kernel(CopyArgs p) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.first[3]; i += (int64_t)gridDim.x * 256) {
        const int o = i >= p.first[2] ? 2 : i >= p.first[1] ? 1 : 0;
        const int64_t at = i - p.first[o], row = at / p.chunks;
        const int kb = (int)(at - row * p.chunks) * 16;
        *(u32x4 *)(p.dst[o] + row * p.ldd + kb) = load_chunk<T>(p.src[o] + row * p.lds[o], kb, p.kbytes);
    }
}

int64_t prod_copy_pitch(int64_t kbytes) {
    const int64_t whole = (kbytes + 127) / 128 * 128;
    return whole + (256 + 512 - whole % 512) % 512;    // an odd multiple of 256 bytes
}

hipError_t prod_aligned_copies(ProdArgs &p, int t, char *ws, hipStream_t s) {
    const int rows[3] = {p.M, p.N, p.B1 ? p.N : 0};
    const void **from[3] = {&p.A, &p.B, &p.B1};
    int64_t *ld[3] = {&p.lda, &p.ldb, &p.ldb1};
    CopyArgs c;
    c.ldd = prod_copy_pitch(p.KB);
    c.kbytes = p.KB;
    c.chunks = (p.KB + 15) / 16;
    c.first[0] = 0;
    for (int i = 0; i < 3; ++i) {
        c.src[i] = (const char *)*from[i];
        c.dst[i] = ws;
        c.lds[i] = *ld[i];
        c.first[i + 1] = c.first[i] + (int64_t)rows[i] * c.chunks;
        if (rows[i] == 0) continue;
        *from[i] = ws;
        *ld[i] = c.ldd;
        ws += (int64_t)rows[i] * c.ldd;
    }
    p.KB = c.chunks * 16;
    const int64_t want = (c.first[3] + 1023) / 1024;
    const unsigned grid = (unsigned)(want < 65536 ? want : 65536);
    if (t == kI8)
        hipLaunchKernelGGL(prod_copy_kernel<kI8>, dim3(grid), dim3(256), 0, s, c);
    else
        hipLaunchKernelGGL(prod_copy_kernel<1>, dim3(grid), dim3(256), 0, s, c);
    return hipGetLastError();
}

}  // namespace tg
