// beam_api.cu -- the C ABI of beam search (declared in include/spark_beam.h):
// argument checks and launches.
#include "beam.h"
#include "checks.h"

using namespace spark;
using namespace spark::checks;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool words(const void* p) { return p != nullptr && aligned4(p); }

int check_beam_ws(const void* ws, size_t bytes) {
  return !ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || bytes < beam::kTotal ? SPARK_ERR_WORKSPACE : SPARK_OK;
}

bool check_groups(int32_t n_groups, int32_t n_beams) {
  return n_beams >= 1 && n_beams <= SPARK_MAX_BEAMS && n_groups >= 1 && n_groups <= SPARK_MAX_BATCH / n_beams;
}

}  // namespace

extern "C" {

size_t spark_beam_workspace_bytes(int32_t n_groups, int32_t n_beams) {
  return check_groups(n_groups, n_beams) ? beam::kTotal : 0;
}

int spark_beam_select(const void* logits, int64_t ld, int32_t dtype, int32_t n_groups, int32_t n_beams, int32_t vocab,
                      const float* score, const int32_t* done, const int32_t* length, int32_t eos, float* new_score,
                      int32_t* token, int32_t* parent, int32_t* new_done, int32_t* keep_len, int32_t* new_len,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (check_dtype(dtype) != SPARK_OK || !logits || !check_groups(n_groups, n_beams) || vocab < 1 || vocab > (1 << 24) ||
      ld < vocab || ld > ((int64_t)1 << 40) || eos < -1 || eos >= vocab)
    return SPARK_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) & (dtype == SPARK_BF16 ? 1u : 3u)) != 0) return SPARK_ERR_INVALID_ARG;
  if (!words(score) || !words(new_score) || !words(token) || !words(parent)) return SPARK_ERR_INVALID_ARG;
  if (!aligned4(done) || !aligned4(new_done) || (eos < 0 && done) || (eos >= 0 && !new_done)) return SPARK_ERR_INVALID_ARG;
  if ((length != nullptr) != (keep_len != nullptr) || (length != nullptr) != (new_len != nullptr) || !aligned4(length) ||
      !aligned4(keep_len) || !aligned4(new_len))
    return SPARK_ERR_INVALID_ARG;
  const int s = check_beam_ws(workspace, workspace_bytes);
  if (s != SPARK_OK) return s;
  beam::Select a = {logits, ld, n_groups, n_beams, vocab, score, done, length, eos, new_score, token, parent, new_done,
                    keep_len, new_len, nullptr, nullptr};
  a.tickets = ws_at<uint32_t>(workspace, beam::kTickets);
  a.part = ws_at<beam::Part>(workspace, beam::kParts);
  return cuda_status(launch_beam_select(a, dtype, (cudaStream_t)stream));
}

int spark_beam_reorder(const int32_t* parent, const int32_t* keep_len, const int32_t* new_len, int32_t n_slots,
                       const spark_beam_state* states, int32_t n_states, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (!words(parent) || check_batch(n_slots) != SPARK_OK || !states || n_states < 1 || n_states > SPARK_MAX_BEAM_STATES)
    return SPARK_ERR_INVALID_ARG;
  if (!aligned4(keep_len) || !aligned4(new_len)) return SPARK_ERR_INVALID_ARG;
  beam::States all = {};
  // what a call writes is nothing that it reads or writes elsewhere
  struct Span {
    uintptr_t begin, end;
    bool meets(const Span& o) const { return begin < o.end && o.begin < end; }
  };
  auto span = [](const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, p ? a + (uintptr_t)bytes : a};
  };
  const Span lists[3] = {span(parent, 4 * (int64_t)n_slots), span(keep_len, 4 * (int64_t)n_slots), span(new_len, 4 * (int64_t)n_slots)};
  for (int i = 0; i < n_states; ++i) {
    const spark_beam_state& t = states[i];
    if (!words(t.src) || !words(t.dst) || t.pitch < 4 || t.pitch % 4 != 0 || t.pitch >= ((int64_t)1 << 31) || t.elem < 0 ||
        t.elem % 4 != 0 || t.elem > t.pitch || !aligned4(t.push) || (t.push && t.elem != 4))
      return SPARK_ERR_INVALID_ARG;
    if (t.elem > 0 && (!keep_len || !new_len)) return SPARK_ERR_INVALID_ARG;
    const Span dst = span(t.dst, n_slots * t.pitch);
    for (const Span& l : lists)
      if (dst.meets(l)) return SPARK_ERR_INVALID_ARG;
    all.s[i] = t;
  }
  for (int i = 0; i < n_states; ++i) {
    const Span dst = span(states[i].dst, n_slots * states[i].pitch);
    for (int j = 0; j < n_states; ++j) {
      const spark_beam_state& o = states[j];
      if (dst.meets(span(o.src, n_slots * o.pitch)) || dst.meets(span(o.push, 4 * (int64_t)n_slots)) ||
          (i != j && dst.meets(span(o.dst, n_slots * o.pitch))))
        return SPARK_ERR_INVALID_ARG;
    }
  }
  const int s = check_beam_ws(workspace, workspace_bytes);
  if (s != SPARK_OK) return s;
  return cuda_status(launch_beam_reorder(parent, keep_len, new_len, n_slots, all, n_states, ws_at<uint32_t>(workspace, 0),
                                         (cudaStream_t)stream));
}

}  // extern "C"
