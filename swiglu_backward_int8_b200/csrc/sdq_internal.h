// Shared by the library's translation units; not part of its interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace sdq_internal {

// Records e for sdq_last_cuda_error and returns SDQ_ERR_CUDA (sdq_api.cu).
int cuda_fail(cudaError_t e);

// The current device's multiprocessors; SDQ_OK or a status (sdq_api.cu).
int sm_count(int* sms);

// The current device's status word, which sdq_device_status reads (sdq_api.cu).
int device_status_word(int** word);

// The limit of a kernel's wait on a barrier, in nanoseconds (sdq_api.cu).
uint64_t wait_limit();

// A row-major [rows, inner] byte array read in boxes of `box_rows` x 128
// bytes, laid out in shared memory with the 128-byte swizzle; bytes out of
// range read as zero (sdq_api.cu).
int make_code_map(CUtensorMap* map, const void* base, uint64_t inner_bytes, uint64_t rows, uint64_t row_bytes,
                  uint32_t box_rows);

// Scale tiles of 512 bytes, `tiles_k` of them side by side for each of `blocks`
// blocks of 128 rows, read `box_tiles` at a time (coordinates in words of 8
// bytes); tiles out of range read as zero (sdq_api.cu).
int make_scale_map(CUtensorMap* map, const void* base, uint64_t tiles_k, uint64_t blocks, uint32_t box_tiles);

// A row-major [rows, cols] array of fp32 or bf16, written in boxes of 32 rows x
// 128 bytes with the 128-byte swizzle; what is out of range is not written
// (sdq_api.cu).
int make_out_map(CUtensorMap* map, void* base, bool f32, uint64_t cols, uint64_t rows, uint64_t ld);

}  // namespace sdq_internal
