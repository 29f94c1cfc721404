// Compiled with a barrier that counts an arrival which does not come and a short limit (built and run by tests/test_gpu_adapter_status.py): each kernel with bounded waits
// ends, says so in the status word, and has written nothing but its results.
#include "adapter_plan.cu"
#include "adapter_sum.cu"

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "adapter_pass.cuh"

using namespace sgb;
using B = __nv_bfloat16;

static_assert(ad::LOST_ROWS + ad::LOST_DONE == 1 && ad::WAIT_NS <= 20000000, "this is a test's build");

static int bad = 0;

static void want(bool ok, const char* what, const char* name)
{
    if (!ok) std::printf("%s: %s\n", name, what), ++bad;
}

static void must(cudaError_t e)
{
    if (e == cudaSuccess) return;
    std::printf("%s\n", cudaGetErrorString(e));
    std::exit(2);
}

// Device memory between two pages of a pattern.
struct Room {
    static constexpr size_t PAGE = 4096;
    size_t bytes;
    uint8_t* at;
    explicit Room(size_t n) : bytes((n + 255) / 256 * 256)
    {
        must(cudaMalloc(&at, bytes + 2 * PAGE));
        must(cudaMemset(at, 0x5a, bytes + 2 * PAGE));
        must(cudaMemset(at + PAGE, 0, bytes));
    }
    ~Room() { must(cudaFree(at)); }
    template <typename T>
    T* as() const { return reinterpret_cast<T*>(at + PAGE); }
    bool whole() const
    {
        std::vector<uint8_t> h(bytes + 2 * PAGE);
        must(cudaMemcpy(h.data(), at, h.size(), cudaMemcpyDeviceToHost));
        for (size_t i = 0; i < PAGE; ++i)
            if (h[i] != 0x5a || h[PAGE + bytes + i] != 0x5a) return false;
        return true;
    }
    bool zero() const
    {
        std::vector<uint8_t> h(bytes);
        must(cudaMemcpy(h.data(), at + PAGE, bytes, cudaMemcpyDeviceToHost));
        for (const uint8_t v : h)
            if (v) return false;
        return true;
    }
};

int main()
{
    Room status(4);
    const auto told = [&](const char* name) {
        uint32_t word = 0;
        must(cudaDeviceSynchronize());
        must(cudaMemcpy(&word, status.as<uint32_t>(), 4, cudaMemcpyDeviceToHost));
        must(cudaMemset(status.as<uint32_t>(), 0, 4));
        want(word == 6u, "no report", name);
    };
    const struct { int64_t rows; int adapters, rank, from, to; } sizes[] = {{300, 2, 16, 1024, 264}, {129, 1, 72, 2048, 136}, {700, 40, 24, 136, 512}};
    for (const auto& z : sizes) {
        std::vector<int> index(z.rows);
        for (int64_t t = 0; t < z.rows; ++t) index[t] = static_cast<int>(t * 7 % z.adapters);
        Room index_dev(z.rows * 4), plan(adapter_plan_bytes(z.rows, z.adapters));
        Room in(z.rows * z.from * 2), w1(size_t(z.adapters) * z.rank * z.from * 2), w2(size_t(z.adapters) * z.rank * z.to * 2), base(z.rows * z.to * 4), out(z.rows * z.to * 4);
        Room mid(z.rows * z.rank * 4), sums(size_t(z.adapters) * z.rank * z.from * 4), part(size_t(2) * ad::PlanLayout(z.rows, z.adapters).tiles * z.rank * z.from * 4);
        must(cudaMemcpy(index_dev.as<int>(), index.data(), z.rows * 4, cudaMemcpyHostToDevice));
        want(adapter_plan(z.rows, z.adapters, index_dev.as<int>(), plan.as<int>(), nullptr) == CONV2D_OK, "plan", "plan");
        ad::PassParams p{};
        p.plan = ad::plan_of(plan.as<int>(), z.rows, z.adapters);
        p.in = in.as<B>(), p.w1 = w1.as<B>(), p.w2 = w2.as<B>(), p.base = base.as<float>(), p.out = out.as<float>(), p.mid = mid.as<float>();
        p.status = status.as<uint32_t>();
        p.in_stride = z.from, p.base_stride = p.out_stride = z.to;
        p.adapters = z.adapters, p.rank = z.rank, p.from = z.from, p.to = z.to;
        for (p.splits = 1; p.splits <= 8; p.splits *= 2) {
            want(ad::start_pass_as<false, true, 0, float, float>(p, nullptr) == CONV2D_OK, "start", "forward");
            told("forward");
            want(ad::start_pass_as<true, false, 1, float, float>(p, nullptr) == CONV2D_OK, "start", "backward, by elements, halved tiles");
            told("backward, by elements, halved tiles");
        }
        for (const int each : {1, 2, 32}) {
            ad::SumParams s{};
            s.plan = p.plan;
            s.status = p.status;
            s.adapters = z.adapters, s.rank = z.rank;
            ad::SumJob& job = s.jobs[0];
            job.in = in.as<B>(), job.mid = mid.as<float>(), job.out = sums.as<float>(), job.part = part.as<float>();
            job.in_stride = job.cols = z.from, job.tiles_each = each, job.out_col = 1;
            for (job.mode = 0; job.mode < 2; ++job.mode) {
                want(ad::launch_sums(s, ad::PlanLayout(z.rows, z.adapters), nullptr) == CONV2D_OK, "start", "sums");
                told("sums");
            }
        }
        for (const Room* r : {&index_dev, &plan, &in, &w1, &w2, &base, &out, &mid, &sums, &part, &status}) want(r->whole(), "written outside", "memory");
        for (const Room* r : {&in, &w1, &w2, &base}) want(r->zero(), "an operand was written", "memory");
    }
    std::printf("%d wrong\n", bad);
    return bad ? 1 : 0;
}
