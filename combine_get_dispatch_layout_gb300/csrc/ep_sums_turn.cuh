// Whose turn a buffer of sums is: what the issuer of the fp8 experts' products waits for before a block's products go
// into TMEM. Plain C++, so that the order can be checked on the host for any sequence of tiles.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define EP_TURN __host__ __device__ __forceinline__
#else
#define EP_TURN inline
#endif

namespace ep {

constexpr int kBuffers = 4;   // of sums in TMEM, 128 columns apart (rows as lanes: two of 256)

// A block of a tile with rows as columns takes the next buffer; one of two groups of warps reads all of it and announces
// that it is done on the buffer's barrier. A block of a tile with rows as lanes takes an even buffer and the next; each
// group reads half of both, and group h announces on the barrier of buffer + h that it is done with its halves.
struct SumsTurn {
    int buffer = 0;
    uint32_t parities = 15;   // a bit for each buffer: of the phase that is waited for (the first round waits for nothing)
    uint32_t halves = 0;      // a bit for the even buffer of each pair that was last read in halves

    // Calls wait(buffer, parity) for what the next block's sums may not overwrite, and returns its buffer.
    template <typename Wait>
    EP_TURN int next(bool lanes, Wait wait) {
        if (lanes) {
            buffer = (buffer + 1) & 2;
            wait(buffer + 1, (parities >> (buffer + 1)) & 1);
            parities ^= 2u << buffer;
            halves |= 1u << buffer;
        } else if ((halves >> buffer) & 1) {   // the other group's half of it: announced on the odd one, whose own turn waits for it again
            wait(buffer + 1, (parities >> (buffer + 1)) & 1);
            halves &= ~(1u << buffer);
        }
        wait(buffer, (parities >> buffer) & 1);
        parities ^= 1u << buffer;
        const int mine = buffer;
        buffer = (buffer + (lanes ? 2 : 1)) % kBuffers;
        return mine;
    }
};

}  // namespace ep
