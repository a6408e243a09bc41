// abi_prompt.h -- what the decoder layer (abi.cu) shares with the prompt entry
// points (abi_prompt.cu).
#pragma once
#include "abi_common.h"
#include "internal.h"

namespace dfl {

// Shapes of a packed prompt attention; context: with cached positions (base_pos).
int check_prompt_shape(const dflash_dims& d, int S, int M, bool context, int max_pos, const dflash_kv& kv,
                       const char* who);
PromptAttnDesc prompt_attn_desc(const dflash_dims& d, int S, int M, bool context, int max_pos, const dflash_kv& kv,
                                float scale);
QkNormDesc qk_norm_desc(const dflash_dims& d, int M, int rows, const dflash_kv* cache);
// Workspace of the prompt ops; 0 on invalid arguments.
size_t prompt_op_workspace(int op, const void* args, const char* who);

}  // namespace dfl
