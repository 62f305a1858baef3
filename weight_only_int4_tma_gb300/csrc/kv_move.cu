// Cached tokens to other slots (include/decode.h).  A thread has one 16-byte piece of the keys or
// values of a slot and takes it through all moves of a group, one after another: no other
// thread touches that piece, so the order holds without any synchronisation.
//
// Up to eight moves' loads go together, as a path's moves are a chain of latencies otherwise: 256 groups of up to
// 12 moves of 4 KB 5.7 us (9.5 one after another in a CUDA graph, 7.2 together; 1.4 for the bytes), one
// group of 4 moves 4.3 us, the call itself.
#include "decode.cuh"

namespace w4g {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 8;

__global__ void __launch_bounds__(kMoveThreads) move_kernel(MoveArgs a, int page_shift) {
    grid_dep_wait();
    const int side = a.kv_heads * a.row_chunks;  // pieces of a slot's keys
    const int piece = static_cast<int>(blockIdx.y) * kMoveThreads + static_cast<int>(threadIdx.x);
    if (piece >= 2 * side) return;
    const KvView& kv = piece < side ? a.kc : a.vc;
    const int p = piece < side ? piece : piece - side;
    const int head = p / a.row_chunks;
    char* base = static_cast<char*>(kv.p) + head * kv.head_stride + 16 * (p - head * a.row_chunks);
    auto at = [&](int64_t slot) {
        const int64_t page = page_shift >= 0 ? slot >> page_shift : slot / a.page_size;
        return reinterpret_cast<uint4*>(base + page * kv.page_stride + (slot - page * a.page_size) * kv.slot_stride);
    };
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int first = a.starts[b], last = a.starts[b + 1];
        if (first < 0 || last < first || last > a.N) {
            record_status(a.status, kDecInvalidArg);
            continue;
        }
        // Eight moves at a time: their loads go together, unless one reads what another of them writes.
        // (Unsigned: the last ones' numbers may pass 2^31 before they are found to be past the end.)
        const unsigned end = static_cast<unsigned>(last);
        for (unsigned i0 = static_cast<unsigned>(first); i0 < end; i0 += kMoveBatch) {
            int64_t src[kMoveBatch], dst[kMoveBatch];
            bool apart = true;
#pragma unroll
            for (int j = 0; j < kMoveBatch; ++j) {
                src[j] = dst[j] = -1;
                if (i0 + j < end) src[j] = a.src[i0 + j], dst[j] = a.dst[i0 + j];
            }
#pragma unroll
            for (int j = 0; j < kMoveBatch; ++j) {
                if (src[j] >= 0 && dst[j] >= 0 && (src[j] >= a.num_slots || dst[j] >= a.num_slots)) {
                    record_status(a.status, kDecInvalidArg);
                    src[j] = -1;
                }
                if (src[j] < 0) dst[j] = -1;
                if (dst[j] < 0) src[j] = -1;
#pragma unroll
                for (int k = 0; k < j; ++k) apart &= src[j] != dst[k] || src[j] < 0;
            }
            uint4 v[kMoveBatch];
            if (apart) {
#pragma unroll
                for (int j = 0; j < kMoveBatch; ++j)
                    if (src[j] >= 0) v[j] = *at(src[j]);
#pragma unroll
                for (int j = 0; j < kMoveBatch; ++j)
                    if (src[j] >= 0) *at(dst[j]) = v[j];
            } else {
#pragma unroll
                for (int j = 0; j < kMoveBatch; ++j)
                    if (src[j] >= 0) *at(dst[j]) = *at(src[j]);
            }
        }
    }
}

}  // namespace

int launch_move(const MoveArgs& a, cudaStream_t stream) {
    const unsigned blocks = blocks_for(2 * a.kv_heads * a.row_chunks, kMoveThreads);
    if (blocks > 65535) return -2;
    return launch_dependent(move_kernel, dim3(static_cast<unsigned>(a.B < 65536 ? a.B : 65536), blocks),
                            dim3(kMoveThreads), 0, stream, a, power_of_two(a.page_size));
}

}  // namespace w4g
