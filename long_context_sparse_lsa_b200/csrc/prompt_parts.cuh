// prompt_parts.cuh — which kernel combines the key parts of whole-prompt attention.
#pragma once

#include <cstdint>

namespace lsa {

// With a token or two per sequence (attend_prompt_few.cu) up to this many parts
// of a row are one cluster (the portable size) and need no workspace.
constexpr int kFewJoined = 8;


// Columns, (row, query head) pairs of a sequence and kv head, that one CTA of
// it takes: those of most sequences are 8 or fewer (one token of up to 8
// heads), or more.
inline int few_columns(int n_seq, int n_rows, int G) { return (int64_t)n_rows * G > (int64_t)n_seq * 8 ? 16 : 8; }

}  // namespace lsa
