// The eps that a step takes, by the states' size: the stand-ins and helpers are
// those of the AdamW step's host checks.
#define main adamw_host_checks_main
#include "adamw_host_checks.cpp"
#undef main

namespace {

void eps_of(bool small)
{
    std::mt19937 rng(9);
    List l(rng, small);
    while (l.numel.empty() || l.numel[0] == 0) l = List(rng, small);   // a list without elements launches nothing
    const size_t bytes = ddp_adamw_workspace_bytes(&l.d);
    Space ws(bytes);
    l.d.workspace = ws.at;
    l.d.workspace_bytes = bytes;
    ddp_adamw *o = nullptr;
    expect(ddp_adamw_create(&l.d, &o) == DDP_OK && o, "eps: create");
    if (!o) return;
    const auto taken = [&](double eps) {
        ddp_adamw_args a = usual();
        a.eps = eps;
        const int before = g_launches, rc = ddp_adamw_step(o, &a, nullptr);
        expect((rc == DDP_OK) == (g_launches == before + 1), "eps: launches");
        return rc == DDP_OK;
    };
    for (double eps : {0.0, 0x1p-126, 1e-8, 1.0, 0x1p125}) expect(taken(eps), "eps refused: " + std::to_string(eps));
    for (double eps : {0x1.000002p125, 0x1p126, 3e38}) expect(taken(eps) == !small, "large eps: " + std::to_string(eps));
    for (double eps : {-1.0, 0x1p-127, 0x1p128}) expect(!taken(eps), "eps taken: " + std::to_string(eps));
    ddp_adamw_destroy(o);
}

}  // namespace

int main()
{
    eps_of(false);
    eps_of(true);
    if (g_bad) return 1;
    std::printf("adamw_eps_checks ok\n");
    return 0;
}
