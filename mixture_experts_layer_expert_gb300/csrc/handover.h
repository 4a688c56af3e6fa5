// handover.h -- bookkeeping of a block's requests for further work items (cluster launch control): one answer, a
// 16-byte asynchronous write into the block's shared memory, completes one phase of one barrier.  Host code too, so that
// it can be tested there.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FS_HD __host__ __device__ __forceinline__
#else
#define FS_HD inline
#endif

namespace fs {

struct HandOver {
    uint32_t asked = 0, answered = 0;      // requests issued, answers waited for with success

    FS_HD void ask() { ++asked; }
    FS_HD void answer() { ++answered; }
    // Whether an answer may still be on its way.  A block must not end before it has landed; where none is, there is
    // nothing to wait for.
    FS_HD bool pending() const { return asked != answered; }
    // Parity of the phase that the oldest answer not waited for completes.
    FS_HD uint32_t parity() const { return answered & 1u; }
};

}  // namespace fs
