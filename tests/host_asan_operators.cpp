// Host-side driver for the AddressSanitizer check of the operators for rounded
// layers: workspace sizes over many shapes, and every call along the paths that
// end on the host (refused arguments).  No call here reaches a HIP runtime
// function.  Exit status 0 when every call returned what the C ABI documents.
#include <bakron.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

static int g_fail = 0;

#define CHECK(cond)                                                                 \
    do {                                                                            \
        if (!(cond)) {                                                              \
            std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
            ++g_fail;                                                               \
        }                                                                           \
    } while (0)

// A refusal leaves a message.
static void refused_at(int line, int32_t status, const char *word) {
    if ((status == BAKRON_ERR_INVALID_ARG || status == BAKRON_ERR_WORKSPACE) &&
        std::strstr(bakron_last_error(), word))
        return;
    std::fprintf(stderr, "call at line %d: status %d, \"%s\"\n", line, status, bakron_last_error());
    ++g_fail;
}
#define refused(...) refused_at(__LINE__, __VA_ARGS__)

static void workspace_sizes() {
    const int64_t sizes[] = {1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000, 4096, 8191, 65536, 1 << 20, 1 << 24};
    const int32_t groups[] = {1, 2, 7, 64, 65, 1000, 4096};
    for (int64_t rows : sizes)
        for (int64_t n : sizes)
            for (int64_t k : sizes)
                for (int32_t g : groups) {
                    const size_t f = bakron_fp8_matmul_workspace_size(rows, n, k, g);
                    const size_t h = bakron_grouped_matmul_workspace_size(rows, n, k, g);
                    // parts are for launches that leave CUs idle: at most a few rounds of tiles
                    CHECK(f <= (size_t(1) << 30) && h <= (size_t(1) << 30));
                }
    for (int64_t rows : sizes)
        for (int64_t vocab : {int64_t(1), int64_t(17), int64_t(4096), int64_t(131073), int64_t(1) << 21})
            for (int32_t k : {0, 1, 20, 64}) {
                const size_t w = bakron_token_logprobs_workspace_size(rows, vocab, k);
                CHECK(w <= (size_t(1) << 30));
            }
    CHECK(bakron_fp8_matmul_workspace_size(0, 1, 1, 1) == 0);
    CHECK(bakron_fp8_matmul_workspace_size(INT64_MAX, INT64_MAX, INT64_MAX, INT32_MAX) == 0);
    CHECK(bakron_grouped_matmul_workspace_size(-1, 1, 1, 1) == 0);
    CHECK(bakron_grouped_matmul_workspace_size(1, 1, INT64_MIN, -1) == 0);
    CHECK(bakron_token_logprobs_workspace_size(0, 1, 0) == 0);
    CHECK(bakron_token_logprobs_workspace_size(INT64_MAX, INT64_MAX, INT32_MAX) == 0);
}

static void refusals() {
    // never read: every call below is refused first
    uint8_t *const p = reinterpret_cast<uint8_t *>(0x10000);
    float *const f = reinterpret_cast<float *>(0x20000);
    int32_t *const off = reinterpret_cast<int32_t *>(0x30000);
    int64_t *const t = reinterpret_cast<int64_t *>(0x40000);
    refused(bakron_fp8_quantize(nullptr, BAKRON_T_F32, 1, 1, 1, 1, p, 1, f, nullptr, nullptr), "NULL");
    refused(bakron_fp8_quantize(f, 9, 1, 1, 1, 1, p, 1, f, nullptr, nullptr), "type");
    refused(bakron_fp8_quantize(f, BAKRON_T_F32, INT64_MAX, 1, 1, 1, p, 1, f, nullptr, nullptr), "sizes");
    refused(bakron_fp8_quantize(f, BAKRON_T_F32, 4, 8, 7, 1, p, 8, f, nullptr, nullptr), "ld");
    refused(bakron_fp8_from_codes(nullptr, nullptr, 1, 1, BAKRON_Q_SYM, 4, p, 1, nullptr), "NULL");
    refused(bakron_fp8_from_codes(reinterpret_cast<int8_t *>(p), nullptr, 1, 1, BAKRON_Q_SYM, 9, p, 1, nullptr), "");
    refused(bakron_fp8_matmul(p, 8, f, p, 8, f, 7, 4, 4, 8, 1, nullptr, p, BAKRON_T_BF16, 4, nullptr, nullptr, 0, nullptr), "scale");
    refused(bakron_fp8_matmul(p, 8, f, p, 8, f, 0, 4, 4, 8, 2, nullptr, p, BAKRON_T_BF16, 4, nullptr, nullptr, 0, nullptr), "offsets");
    refused(bakron_fp8_matmul(p, 8, f, p, 8, f, 0, 4, 4, INT64_MAX, 1, nullptr, p, BAKRON_T_BF16, 4, nullptr, nullptr, 0, nullptr), "sizes");
    refused(bakron_fp8_matmul(p, INT64_MAX, f, p, 8, f, 0, 4, 4, 8, 1, nullptr, p, BAKRON_T_BF16, 4, nullptr, nullptr, 0, nullptr), "ldx");
    for (auto call : {bakron_grouped_matmul, bakron_grouped_matmul_grad_x, bakron_grouped_matmul_grad_w}) {
        refused(call(p, BAKRON_T_BF16, 64, p, 64, 4, 64, 64, 2, off, nullptr, BAKRON_T_BF16, 64, nullptr, nullptr, 0, nullptr), "NULL");
        refused(call(p, BAKRON_T_F32, 64, p, 64, 4, 64, 64, 2, off, p, BAKRON_T_F32, 64, nullptr, nullptr, 0, nullptr), "type");
        refused(call(p + 1, BAKRON_T_BF16, 64, p, 64, 4, 64, 64, 2, off, p, BAKRON_T_BF16, 64, nullptr, nullptr, 0, nullptr), "misaligned");
        refused(call(p, BAKRON_T_BF16, 64, p, 64, 1 << 24, 1 << 24, 1 << 24, 2, off, p, BAKRON_T_BF16, 64, nullptr, nullptr, 0, nullptr), "tiles");
        refused(call(p, BAKRON_T_BF16, 64, p, 64, 4, 64, 64, INT32_MAX, off, p, BAKRON_T_BF16, 64, nullptr, nullptr, 0, nullptr), "groups");
    }
    // no workspace, and one off its alignment
    const size_t need = bakron_fp8_matmul_workspace_size(128, 4096, 4096, 1);
    CHECK(need > 0);
    refused(bakron_fp8_matmul(p, 4096, f, p, 4096, f, 0, 128, 4096, 4096, 1, nullptr, p, BAKRON_T_BF16, 4096, nullptr, nullptr, need, nullptr), "workspace");
    refused(bakron_fp8_matmul(p, 4096, f, p, 4096, f, 0, 128, 4096, 4096, 1, nullptr, p, BAKRON_T_BF16, 4096, nullptr, p + 128, need, nullptr), "workspace");
    refused(bakron_token_logprobs(nullptr, 0, 1, 1, 1, t, 0, f, f, f, nullptr, nullptr, nullptr, nullptr, 0, nullptr), "NULL");
    refused(bakron_token_logprobs(f, 0, 1, INT64_MAX, 1, t, 0, f, f, f, nullptr, nullptr, nullptr, nullptr, 0, nullptr), "sizes");
    refused(bakron_token_logprobs(f, 0, 1, 100, 100, t, 65, f, f, f, f, t, nullptr, nullptr, 0, nullptr), "k");
    refused(bakron_token_logprobs_grad(f, 0, 1, 100, 99, t, f, f, f, f, f, 100, nullptr, nullptr), "ld");
}

int main() {
    workspace_sizes();
    refusals();
    if (g_fail) return 1;
    std::puts("host checks passed");
    return 0;
}
