// abi_tree.h -- what the decoder layer (abi.cu) shares with the tree
// verification entry points (abi_tree.cu).
#pragma once
#include "abi_common.h"
#include "internal.h"

namespace dfl {

int check_tree_shape(const dflash_dims& d, int S, int rows, int max_pos, const dflash_kv& kv, const char* who);
int check_tree_kv(const dflash_kv& kv, const char* who);
TreeAttnDesc tree_attn_desc(const dflash_dims& d, int S, int rows, int max_pos, const dflash_kv& kv, float scale);
// Workspace of the tree verification ops; 0 on invalid arguments.
size_t tree_op_workspace(int op, const void* args, const char* who);

}  // namespace dfl
