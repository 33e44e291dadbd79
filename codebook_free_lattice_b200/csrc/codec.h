// codec.h -- the codec object behind the C ABI's opaque handle, and what the library's translation
// units share about it (llvq.cu: decode, encode, products, search; linear.cu: linear layers).
#pragma once
#include <atomic>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string>

#include "../../include/llvq.h"
#include "codec72.cuh"
#include "codec96.cuh"
#include "tables.h"

struct llvq_codec {
    int index_bits = 0;
    int device = -1;
    int M = 0;
    llvq::u128 npoints = 0;
    int64_t nclasses = 0;
    int num_sms = 0;
    void *d_image = nullptr;       // Smem48 / Smem72 image (copied to shared memory per CTA)
    llvq::Rec72 *d_recs72 = nullptr;     // 72-bit class records (global memory)
    uint32_t *d_guide72 = nullptr; // 72-bit guide table
    llvq::Rec96 *d_recs96 = nullptr;     // 96-bit class records (global memory)
    uint32_t *d_guide96 = nullptr; // 96-bit guide table (top 28 index bits)
    void *d_even48 = nullptr;      // SmemEven48 image (48-bit table path)
    uint32_t *d_tabC48 = nullptr;  // complement arrangement tables (48-bit table path)
    void *d_gv48 = nullptr;        // SmemGv48 image (48-bit fused products, k_gemv48)
    void *d_enc48 = nullptr;       // EncSmem48 image (48-bit encoder)
    void *d_search48 = nullptr;    // SearchImage48 (48-bit nearest-point search)
    void *d_enc72 = nullptr;       // EncSmem72 image (72-bit encoder)
    unsigned long long *d_keys72 = nullptr;  // 72-bit class keys (encoder)
    void *d_enc96 = nullptr;       // EncSmem96 image (96-bit encoder)
    unsigned long long *d_keys96 = nullptr;  // 96-bit class keys (encoder, built on the device)
    unsigned *d_flags = nullptr;   // sticky device flags
    int pairs = 0;                 // CTA pairs of the linear layers' product that run at once
};

namespace llvq {
extern thread_local std::string g_last_error;
extern std::atomic<uint32_t> g_first_wait_tries, g_mma_wait_tries;
// argument checks of a compressed weight (llvq.cu)
llvq_status check_weight(const llvq_codec *c, const llvq_weight *w);
// shared-memory limits of the linear layers' kernels and pairs, on the codec's device (linear.cu)
cudaError_t set_linear_attrs(llvq_codec *c);
}  // namespace llvq
