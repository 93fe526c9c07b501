"""Two tenants adapt one binarized projection to a float teacher, then share it.

A float projection W (the teacher) is binarized and packed once. Its outputs
serve as logits. For two tenants, whose teachers differ from W by a low-rank
change, adapters beside the packed weights are trained by distillation from
the teachers' top logits, both in one batch:

    forward    bt_binary_linear -> bt_adapter_linear (onto its result)
    loss       bt_distill_topk_step (loss and gradient of the logits)
    backward   bt_binary_linear_backward (the projection's input gradient)
               -> bt_adapter_linear_backward (added to it; the adapters' gradients)

Then a decoding batch of both tenants, and of a request without an adapter,
goes through the same packed weights in one call each.

    python examples/adapter_distillation.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import xnor_popcount_gemm_gb300 as bt  # noqa: E402

K, V, R, TENANTS, SLOTS, TAU = 512, 4096, 16, 2, 64, 2.0


def main(steps: int = 60, tokens: int = 1024, verbose: bool = True) -> tuple[float, float]:
    """Trains for some steps; returns the mean loss before and after."""
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev).manual_seed(0)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * std

    w = normal(V, K, std=K ** -0.5)
    teachers = [w + normal(V, 4, std=0.5) @ normal(4, K, std=K ** -0.5) for _ in range(TENANTS)]
    code, _ = bt.bt_plan(bt.BT_OP_LINEAR, tokens, V, K)
    packed, wst = bt.bt_pack_sign(w, code), bt.bt_sign_transpose(w)
    scale_a, scale_w = 0.8, float(w.abs().mean())

    # adapters: B starts at zero, so that nothing changes before the first step
    a, b = normal(TENANTS, R, K, std=K ** -0.5), torch.zeros(TENANTS, V, R, device=dev)
    scale = torch.ones(TENANTS, device=dev)
    moments = [(torch.zeros_like(p), torch.zeros_like(p)) for p in (a, b)]
    ids = [i * TENANTS // tokens for i in range(tokens)]          # one sequence of each tenant
    plan = bt.bt_adapter_plan(ids, TENANTS, device=dev)
    upstream = torch.full((tokens,), TAU * TAU / tokens, device=dev)

    means = []
    for step in range(steps):
        x = normal(tokens, K).bfloat16()
        teacher = torch.cat([x[i * tokens // TENANTS:(i + 1) * tokens // TENANTS].float() @ teachers[i].t() for i in range(TENANTS)])
        top, slots = teacher.topk(SLOTS, dim=1)                   # what a stored teacher gives
        lse = torch.logsumexp(teacher / TAU, dim=1)

        ab, bb = a.bfloat16(), b.bfloat16()
        base = bt.bt_binary_linear(x, packed, code, K, scale_a, scale_w)
        u = torch.empty(tokens, R, device=dev)
        logits = bt.bt_adapter_linear(x, ab, bb, scale, plan, base=base, out=base, u=u)
        loss, grad = bt.bt_distill_topk_step(upstream, logits, slots, top, lse, TAU, grad=logits)
        gx, _, _ = bt.bt_binary_linear_backward(x, wst, grad, scale_a, scale_w, grad_weight_dtype=None)
        _, ga, gb = bt.bt_adapter_linear_backward(x, grad, u, ab, bb, scale, plan, grad_base=gx, grad_x=gx)

        for p, g, (m, v) in zip((a, b), (ga, gb), moments):       # Adam
            m.mul_(0.9).add_(g, alpha=0.1)
            v.mul_(0.99).addcmul_(g, g, value=0.01)
            k = step + 1
            p.addcdiv_(m / (1 - 0.9 ** k), (v / (1 - 0.99 ** k)).sqrt_().add_(1e-12), value=-1e-2)
        means.append(loss.mean())
        if verbose and (step % 10 == 0 or step == steps - 1):
            print(f"step {step:3d}  loss {means[-1].item():.4f}")

    # decoding: requests of both tenants and one without an adapter, in any order
    x = normal(5, K).bfloat16()
    served = bt.bt_adapter_plan([1, 0, -1, 1, 0], TENANTS, device=dev)
    base = bt.bt_binary_linear(x, packed, code, K, scale_a, scale_w)
    logits = bt.bt_adapter_linear(x, a.bfloat16(), b.bfloat16(), scale, served, base=base)
    assert torch.equal(logits[2], base[2]) and not torch.equal(logits[0], base[0])
    assert bt.bt_device_status() == bt.BT_OK
    if verbose:
        print("next tokens:", logits.argmax(dim=1).tolist())
    return means[0].item(), means[-1].item()


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
