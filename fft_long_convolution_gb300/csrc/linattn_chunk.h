// Launch of the linear attention's chunked kernels (linattn_chunk.cu).
#pragma once
#include "delta_chunk.h"
#include "linattn.h"

namespace fftconv {

// A walk over sequences (linattn.h), its tensors as boxes of 64 tokens x 64 features,
// and where the segments' states are: float32 [state][H][DK][DV] of the walk that formed
// them; they are read as w.turned says.  A sequence of n segments has n - 1 of them, in
// the order of time, from its first chunk slot / seg_chunks on: as sequences' chunk slots
// do not meet, neither do these.
struct Pass {
    CUtensorMap mq, mk, mv, mo;
    Walk w;
    float* seg_state;
};

constexpr int kSorted = 32;

// Up to three walks of the same sizes, side by side.
struct Passes {
    Pass p[3];
    int64_t seg_chunks;
    int64_t segments;
    int join;            // a walk's CTAs join the states of sequences of up to so many segments themselves
    int64_t most;        // segments that a sequence may have: past join, the join is launched
    bool few_cut;        // few sequences are cut: their end states' walk looks for those
    bool longest_first;  // packed sequences (up to kSorted), in the order of their lengths
    int* err;
};

// Chunks of a segment, how many segment slots there are (nseq: no sequence is cut) and
// states at segments' ends, for `walks` walks at once.  join: the most segments of a sequence whose states the
// walks' CTAs add up themselves; most: segments that a sequence may have.  few_cut: only
// the long sequences of a packed row are.  by_length: packed sequences in the order of
// their lengths.
struct Segments {
    int64_t chunks, count, states, most;
    int join;
    bool few_cut, by_length;
};
void plan_segments(Segments* s, int64_t B, int64_t T, int64_t nseq, int64_t heads, int walks, int dt, int sms);

// states: the end states of all segments of sequences that are cut (of a walk's last one
// where the final state is wanted), joined along each sequence of more than a.join.
cudaError_t launch_linattn(const Passes& a, int n, bool states, int dt, int dk, int dv, cudaStream_t st);

}  // namespace fftconv
