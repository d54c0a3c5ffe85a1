// row_cut.h -- a row of V elements of an array whose rows lie one behind the other, cut into whole
// vectors of VEC elements, at their places in the array, and the elements beside them ("edges").
#pragma once

#include <stddef.h>

// Vectors f0 .. f1 - 1, counted from the one that holds the row's first element, lie in the row as a
// whole; `mis` elements of the array lie before the row in that one.  Columns 0 .. head - 1 and
// tail .. V - 1 are in none of them: fewer than two vectors' elements.  A row that lies inside one
// vector and does not begin it has no vector of its own, and all of its columns are before the next
// one: the end of the row, not that vector's place, is then where the tail begins.
struct RowCut {
    int mis, f0, f1, head, tail;
};

template <int VEC>
__host__ __device__ inline RowCut cut_row(size_t first, int V)
{
    RowCut r;
    r.mis = (int)(first % VEC);
    r.f0 = r.mis > 0 ? 1 : 0;
    r.f1 = (r.mis + V) / VEC > r.f0 ? (r.mis + V) / VEC : r.f0;
    r.head = r.mis == 0 ? 0 : V < VEC - r.mis ? V : VEC - r.mis;
    r.tail = r.f1 * VEC - r.mis;
    r.tail = r.tail > V ? V : r.tail > r.head ? r.tail : r.head;
    return r;
}
