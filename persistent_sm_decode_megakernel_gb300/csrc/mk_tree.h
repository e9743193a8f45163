// Where the nodes of drafted trees go, for the decoder's step over them.
#pragma once
#include "../../include/mk.h"

namespace mk {

// Of every node of n_rows trees: its position (lens + its ancestors; -1 where it is absent), its slot (lens + its
// number) and its table row, device int32 [n_rows][n_nodes] each.  rows NULL: row r.
mk_status tree_places(const int32_t* lens, const int32_t* parents, const int32_t* rows, int n_rows, int n_nodes, int32_t* positions,
                      int32_t* slots, int32_t* table_rows, void* stream);

}  // namespace mk
