// Launchers of rotary positions outside the cache (rope.hip).
#pragma once

#include "kronq_internal.h"

namespace kronq {

struct HeadsView;
struct RopeView;

constexpr int kRopePairs = 256;           // of a table: they travel as a kernel's argument

// The dim / 2 frequencies, in fp64 (host).
void rope_frequencies(const kronq_rope_scaling& c, int dim, double* f);

// Workgroups of a call's launch, for the checks of their number.
int64_t rope_tables_grid(int64_t positions, int dim);
int64_t rotate_grid(int64_t rows, int64_t heads, int dim, int32_t dtype);

kronq_status rope_tables_launch(float* cos, float* sin, int64_t ld, int64_t first, int64_t positions, int dim,
                                const kronq_rope_scaling& c, hipStream_t s);

// in, out, heads: of queries and of keys (0 heads: none)
kronq_status rotate_launch(const HeadsView* in, const HeadsView* out, const int* heads, int32_t dtype, int64_t rows,
                           int dim, const int32_t* pos, const RopeView& r, int back, hipStream_t s);

}  // namespace kronq
