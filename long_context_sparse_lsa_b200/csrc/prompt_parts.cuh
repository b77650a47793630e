// prompt_parts.cuh — which kernel combines the key parts of whole-prompt attention.
#pragma once

namespace lsa {

// With a token or two per sequence (attend_prompt_few.cu) up to this many parts
// of a row are one cluster (the portable size) and need no workspace.
constexpr int kFewJoined = 8;

}  // namespace lsa
