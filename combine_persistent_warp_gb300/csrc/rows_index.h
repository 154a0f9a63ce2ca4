// rows_index.h -- index arithmetic of the row kernels (rows.cu) that keeps their accesses inside the
// tensors, in plain C++ so that it is checked exhaustively on the host too.
#pragma once

#ifdef __CUDACC__
#define CPW_HD __host__ __device__ __forceinline__
#else
#define CPW_HD inline
#endif

namespace cpw {

// First of the rows that no slot has: offsets[E] inside [0, M], whatever it holds, so that a
// grid's strides from there on stay in 31 bits.
CPW_HD int rest_begin(int total, int M) { return total < 0 ? 0 : total > M ? M : total; }

// ------------------------------------------------------------------ rows of any alignment ----
// Rows in the aligned vectors of V elements of their own place: vector g starts at element
// g * V - lead of the row, lead < V.
// vectors that a row of H elements may touch
CPW_HD int vectors_of(int H, int V) { return (H + V - 1 + V - 1) / V; }
// The aligned vectors of elements e .. e + V - 1 of a row lie inside the row, for every e that
// vector g has whatever the row's lead.
CPW_HD bool inside(int g, int H, int V) { return g >= 2 && (g + 2) * V <= H; }
// Row r of `rows` has as many elements of its matrix before and after it as those vectors may reach past
// its ends, whatever the leads (rim: rows that hold them).  A row's first vector starts at element -(V - 1)
// at least, and the aligned ones up to V - 1 before that: 2 V - 2.  Its last one starts at H + V - 2 at most
// (H past a multiple of V by 2, no lead) and takes two aligned ones from there: 3 V - 2 past the end.
CPW_HD bool amid(int r, int rows, int rim) { return r >= rim && r < rows - rim; }
CPW_HD int rim_of(int H, int V) { return (3 * V - 2 + H - 1) / H; }

}  // namespace cpw
