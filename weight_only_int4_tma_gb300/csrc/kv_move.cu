// Cached tokens to other slots (include/decode.h).  A thread has one 16-byte piece of the keys or
// values of a slot and takes it through all moves of a group, one after another: no other
// thread touches that piece, so the order holds without any synchronisation.
#include "decode.cuh"

namespace w4g {
namespace {

constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) move_kernel(MoveArgs a) {
    grid_dep_wait();
    const int side = a.kv_heads * a.row_chunks;  // pieces of a slot's keys
    const int piece = static_cast<int>(blockIdx.y) * kMoveThreads + static_cast<int>(threadIdx.x);
    if (piece >= 2 * side) return;
    const KvView& kv = piece < side ? a.kc : a.vc;
    const int p = piece < side ? piece : piece - side;
    const int head = p / a.row_chunks;
    char* base = static_cast<char*>(kv.p) + head * kv.head_stride + 16 * (p - head * a.row_chunks);
    auto at = [&](int64_t slot) {
        const int64_t page = slot / a.page_size;
        return reinterpret_cast<uint4*>(base + page * kv.page_stride + (slot - page * a.page_size) * kv.slot_stride);
    };
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int first = a.starts[b], last = a.starts[b + 1];
        if (first < 0 || last < first || last > a.N) {
            record_status(a.status, kDecInvalidArg);
            continue;
        }
        for (int i = first; i < last; ++i) {
            const int64_t src = a.src[i], dst = a.dst[i];
            if (src < 0 || dst < 0) continue;
            if (src >= a.num_slots || dst >= a.num_slots) {
                record_status(a.status, kDecInvalidArg);
                continue;
            }
            *at(dst) = *at(src);
        }
    }
}

}  // namespace

int launch_move(const MoveArgs& a, cudaStream_t stream) {
    const unsigned blocks = blocks_for(2 * a.kv_heads * a.row_chunks, kMoveThreads);
    if (blocks > 65535) return -2;
    return launch_dependent(move_kernel, dim3(static_cast<unsigned>(a.B < 65536 ? a.B : 65536), blocks),
                            dim3(kMoveThreads), 0, stream, a);
}

}  // namespace w4g
