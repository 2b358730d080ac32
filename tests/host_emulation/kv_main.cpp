// Bounds-checked CPU run of the key-value cache kernels
// (post_weight_quantization_17_amd/csrc/kv_cache.hip and kv_attention.hip,
// compiled here against the host emulation headers with AddressSanitizer).
// Test infrastructure: tests/test_kv_cache_host.py builds it and compares its
// outputs with a plain implementation.
//
//   kv_host <dir>
//
// <dir>/args.txt: op n_pages page_size kv_heads head_dim bits max_pages ld_table
//   batch n_tokens starts q_heads dtype out_dtype ld ld_out offset scale slopes prompt_min_rows
//   op: write, read or attend; starts, slopes: 0 or 1; ld, ld_out: token
//   strides of the dense inputs and outputs; offset: elements by which the
//   dense buffers are shifted inside their allocations; prompt_min_rows: query
//   rows from which on attend runs the prompts' kernel, -1: the entry point's
//   own rule (which asks for more than a CPU run can hold).
// Inputs (.bin): k_codes v_codes k_grid v_grid table lens [starts], and k v or
// q [slopes]; outputs: the cache's buffers after a write, k_out v_out or out
// (filled with 0xA5 bytes beforehand), info. Every buffer is its own
// allocation of exactly its size.
#include "../../post_weight_quantization_17_amd/csrc/kv_cache.hip"
#include "../../post_weight_quantization_17_amd/csrc/kv_attention.hip"
#include "../../post_weight_quantization_17_amd/csrc/kv_prompt.hip"

#include <fstream>
#include <string>

namespace {

std::string dir;

struct Buf {
  char* base = nullptr;
  size_t bytes = 0, shift = 0;
  char* at() const { return base + shift; }
  template <typename T>
  T* as() const {
    return reinterpret_cast<T*>(base + shift);
  }
};
std::vector<char*> owned;
// An allocation of exactly n + shift bytes, 256-byte aligned.
Buf make(size_t n, size_t shift = 0) {
  void* p = nullptr;
  if (posix_memalign(&p, 256, n + shift ? n + shift : 1) != 0) std::abort();
  std::memset(p, 0xA5, n + shift);
  owned.push_back(static_cast<char*>(p));
  return Buf{static_cast<char*>(p), n, shift};
}
Buf slurp(const char* name, size_t shift = 0) {
  std::ifstream f(dir + "/" + name + ".bin", std::ios::binary);
  const std::vector<char> v((std::istreambuf_iterator<char>(f)), std::istreambuf_iterator<char>());
  Buf b = make(v.size(), shift);
  std::memcpy(b.at(), v.data(), v.size());
  return b;
}
void spill(const char* name, const Buf& b) {
  std::ofstream f(dir + "/" + name + ".bin", std::ios::binary);
  f.write(b.at(), std::streamsize(b.bytes));
}

}  // namespace

int main(int argc, char** argv) {
  if (argc != 2) return 2;
  dir = argv[1];
  char op[16];
  long long n_pages, page_size, kv_heads, head_dim, max_pages, ld_table, batch, n_tokens, q_heads, ld, ld_out;
  int bits, starts, dtype, out_dtype, offset, slopes;
  long long min_rows;
  double scale;
  {
    FILE* f = std::fopen((dir + "/args.txt").c_str(), "r");
    if (!f || std::fscanf(f, "%15s %lld %lld %lld %lld %d %lld %lld %lld %lld %d %lld %d %d %lld %lld %d %lf %d %lld", op,
                          &n_pages, &page_size, &kv_heads, &head_dim, &bits, &max_pages, &ld_table, &batch, &n_tokens,
                          &starts, &q_heads, &dtype, &out_dtype, &ld, &ld_out, &offset, &scale, &slopes, &min_rows) != 20)
      return 2;
    std::fclose(f);
  }
  const Buf kc = slurp("k_codes"), vc = slurp("v_codes"), kg = slurp("k_grid"), vg = slurp("v_grid"),
            table = slurp("table"), lens = slurp("lens");
  const gptq_kv_cache cache{kc.as<uint32_t>(), vc.as<uint32_t>(), kg.as<uint32_t>(), vg.as<uint32_t>(), n_pages,
                            page_size, kv_heads, head_dim, bits};
  Buf st{};
  if (starts) st = slurp("starts");
  const gptq_kv_batch b{table.as<int32_t>(), ld_table, max_pages, lens.as<int32_t>(),
                        starts ? st.as<int32_t>() : nullptr, batch, n_tokens};
  Buf info = make(4);
  *info.as<int32_t>() = 0;
  const size_t eb = gptq::kv_elem_bytes(dtype), eo = gptq::kv_elem_bytes(out_dtype);
  const std::string o = op;
  int rc;
  if (o == "write") {
    const Buf k = slurp("k", offset * eb), v = slurp("v", offset * eb);
    rc = gptq_kv_cache_write(&cache, &b, k.at(), v.at(), dtype, ld, ld, info.as<int32_t>(), nullptr);
    spill("k_codes_out", kc);
    spill("v_codes_out", vc);
    spill("k_grid_out", kg);
    spill("v_grid_out", vg);
  } else if (o == "read") {
    const size_t n = n_tokens ? size_t((n_tokens - 1) * ld_out + kv_heads * head_dim) * eo : 0;
    const Buf k = make(n, offset * eo), v = make(n, offset * eo);
    rc = gptq_kv_cache_read(&cache, &b, k.at(), v.at(), out_dtype, ld_out, ld_out, info.as<int32_t>(), nullptr);
    spill("k_out", k);
    spill("v_out", v);
  } else {
    const Buf q = slurp("q", offset * eb);
    Buf sl{};
    if (slopes) sl = slurp("slopes");
    const Buf out = make(n_tokens ? size_t((n_tokens - 1) * ld_out + q_heads * head_dim) * eo : 0, offset * eo);
    const int64_t from = min_rows < 0 ? gptq::PROMPT_MIN_ROWS : min_rows;
    const size_t wsb = min_rows < 0 ? gptq_kv_attention_workspace_size(&cache, &b, q_heads)
                                    : gptq::attention_workspace(&cache, &b, q_heads, from);
    const Buf ws = make(wsb);
    std::memset(ws.at(), 0xFF, wsb);  // NaN: a partial sum that was not written shows
    const float* sp = slopes ? sl.as<float>() : nullptr;
    void* wp = wsb ? ws.at() : nullptr;
    rc = min_rows < 0 ? gptq_kv_attention(&cache, &b, q.at(), dtype, q_heads, ld, scale, sp, out.at(), out_dtype, ld_out, wp,
                                          wsb, info.as<int32_t>(), nullptr)
                      : gptq::attention(&cache, &b, q.at(), dtype, q_heads, ld, scale, sp, out.at(), out_dtype, ld_out, wp,
                                        wsb, info.as<int32_t>(), nullptr, from);
    spill("out", out);
  }
  spill("info", info);
  for (char* p : owned) std::free(p);
  if (rc != GPTQ_OK) std::fprintf(stderr, "kv_host: status %d\n", rc);
  return rc == GPTQ_OK ? 0 : 3;
}
