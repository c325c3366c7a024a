// Host-side driver for the AddressSanitizer check of rows by group, adapters and draft
// verification: workspace sizes over many shapes, and every call along the paths that end on
// the host (refused arguments), from several threads at once.  No call here reaches a HIP
// runtime function.  Exit status 0 when every call returned what the C ABI documents.
#include <bakron.h>

#include <atomic>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <thread>
#include <vector>

static std::atomic<int> g_fail{0};

#define CHECK(cond)                                                                 \
    do {                                                                            \
        if (!(cond)) {                                                              \
            std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
            ++g_fail;                                                               \
        }                                                                           \
    } while (0)

// A refusal leaves a message.
static void refused_at(int line, int32_t status, const char *word) {
    if ((status == BAKRON_ERR_INVALID_ARG || status == BAKRON_ERR_WORKSPACE) && std::strstr(bakron_last_error(), word)) return;
    std::fprintf(stderr, "call at line %d: status %d, \"%s\"\n", line, status, bakron_last_error());
    ++g_fail;
}
#define refused(...) refused_at(__LINE__, __VA_ARGS__)

static void workspace_sizes() {
    const int64_t sizes[] = {1, 2, 15, 16, 17, 255, 256, 257, 1000, 4096, 8191, 65536, 1 << 20, 1 << 24, INT64_MAX, -1, 0};
    for (int64_t n : sizes)
        for (int32_t g : {-1, 0, 1, 64, 1024, 1025, 4096, 4097, INT32_MAX}) {
            CHECK(bakron_group_sort_workspace_size(n, g) <= (size_t(1) << 28));
            CHECK(bakron_verify_drafts_workspace_size(n, g, 50001) <= (size_t(1) << 20));
            CHECK(bakron_verify_drafts_workspace_size(7, 3, n) <= (size_t(1) << 20));
        }
    for (int64_t rows : sizes)
        for (int64_t n : sizes)
            for (int64_t k : sizes)
                for (int32_t rank : {-1, 1, 16, 100, 256, 257})
                    for (int32_t g : {0, 1, 65, 4096}) {
                        const size_t f = bakron_adapter_matmul_workspace_size(rows, n, k, rank, g);
                        const size_t b = bakron_adapter_matmul_grad_workspace_size(rows, n, k, rank, g);
                        const bool in = rows >= 1 && n >= 1 && k >= 1 && rank >= 1 && rank <= 256 && g >= 1;
                        CHECK(in || (f == 0 && b == 0));
                        CHECK(f <= (size_t(1) << 37));
                    }
}

static void refusals() {
    // never read: every call below is refused first
    void *const p = reinterpret_cast<void *>(0x10000);
    auto *const i32 = static_cast<int32_t *>(p);
    auto *const i64 = static_cast<int64_t *>(p);
    auto *const f32 = static_cast<float *>(p);
    auto *const u8 = static_cast<uint8_t *>(p);
    refused(bakron_group_sort(nullptr, 64, 8, 4, i32, i32, i32, nullptr, nullptr, 0, nullptr), "non-NULL");
    refused(bakron_group_sort(p, 8, 8, 4, i32, i32, i32, nullptr, nullptr, 0, nullptr), "id_bits");
    refused(bakron_group_sort(p, 64, INT64_MAX, 4, i32, i32, i32, nullptr, nullptr, 0, nullptr), "size");
    refused(bakron_group_sort(p, 64, 1 << 20, 4, i32, i32, i32, nullptr, nullptr, 0, nullptr), "workspace");
    refused(bakron_group_gather(p, 1, INT64_MAX, 64, 64, 64, i32, 4, i32, p, 64, nullptr, nullptr), "sizes");
    refused(bakron_group_gather(p, 1, 8, 2, 64, 64, i32, 4, nullptr, p, 64, nullptr, nullptr), "non-NULL");
    refused(bakron_group_gather_fp8(p, 9, 8, 2, 64, 64, i32, 4, i32, u8, 64, f32, nullptr, nullptr), "type");
    refused(bakron_group_combine(p, 1, 8, 2, 64, INT64_MIN, i32, 4, i32, nullptr, p, 64, nullptr, nullptr), "ldy");
    refused(bakron_group_combine_grad(p, 64, p, 1, 8, 2, 64, 64, i32, 4, i32, f32, p, INT64_MAX, f32, nullptr, nullptr), "lddy");
    refused(bakron_adapter_matmul(p, 1, 64, p, p, INT64_MAX, INT64_MAX, 64, 8, 4, i32, i32, f32, p, 64, p, 1, 64, nullptr, p, 0,
                                  nullptr), "sizes");
    refused(bakron_adapter_matmul(p, 1, 64, p, p, 8, 64, 64, INT32_MAX, 4, i32, i32, f32, p, 64, p, 1, 64, nullptr, p, 0, nullptr),
            "rank");
    refused(bakron_adapter_matmul(p, 1, 64, p, p, 8, 64, 64, 8, 4, i32, i32, f32, p, 64, p, 1, 64, nullptr, p, 0, nullptr),
            "workspace");
    refused(bakron_adapter_matmul_grad(p, 64, p, 1, 64, p, p, 8, 64, 64, 8, 4, i32, i32, f32, nullptr, 0, nullptr, 0, 0, p, nullptr,
                                       1, nullptr, p, 0, nullptr), "non-NULL");
    refused(bakron_adapter_matmul_grad(p, 64, p, 1, 64, p, p, 8, 64, 64, 8, 4, i32, i32, f32, nullptr, 0, p, 1, 64, p, p, 1,
                                       nullptr, p, 0, nullptr), "workspace");
    refused(bakron_verify_drafts(p, 64, p, 64, 0, 8, 65, 64, i64, f32, f32, i32, i64, nullptr, p, 0, nullptr), "sizes");
    refused(bakron_verify_drafts(p, 63, p, 64, 0, 8, 4, 64, i64, f32, f32, i32, i64, nullptr, p, 0, nullptr), "ldp");
    refused(bakron_verify_drafts(p, 1 << 17, p, 1 << 17, 0, 1, 4, 1 << 17, i64, f32, f32, i32, i64, nullptr, p, 0, nullptr),
            "workspace");
}

int main() {
    workspace_sizes();
    std::vector<std::thread> threads;
    for (int t = 0; t < 4; ++t) threads.emplace_back([] {
            for (int i = 0; i < 50; ++i) refusals();
        });
    for (auto &t : threads) t.join();
    if (g_fail) return 1;
    std::puts("host checks passed");
    return 0;
}
