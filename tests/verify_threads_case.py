"""Child process of tests/test_verify_threads_gpu.py: the first launches of a verify kernel in a fresh process come from
four host threads at once that ask for different amounts of its shared memory.  Exit status 0 if every call was accepted
and gave the bits of the same call made alone."""
import sys
import threading

import torch

import gated_deltanet_verify_gb300 as gdn
from tests.gpu_util import dims_of, params_of, upload
from workloads.device import empty_outputs
from workloads.synth import Shape, make_inputs

TOKENS = [64, 1, 48, 2]


def main():
    torch.cuda.set_device(0)
    for act in ("bf16", "f32"):
        for d in (32, 64, 128):
            shapes = [Shape(f"vt_{act}_{d}_{T}", n_slots=1, n_qk_heads=2, n_v_heads=4, d_k=d, d_v=d, n_tokens=T, act=act,
                            seed=d + T) for T in TOKENS]
            streams = [torch.cuda.Stream() for _ in shapes]
            sets = [[(upload(make_inputs(s)), empty_outputs(s, "cuda")) for s in shapes] for _ in range(2)]
            torch.cuda.synchronize()
            for mode in ("chain", "lazy"):
                start, errors = threading.Barrier(len(shapes)), []

                def call(i, k):
                    s, (x, o) = shapes[i], sets[k][i]
                    if mode == "chain":
                        gdn.gdn_verify_forward(dims_of(s), params_of(x), x["qkv"], x["z"], x["alpha"], x["beta_raw"],
                                               x["state"], x["conv_state"], o["cap_state"], o["cap_conv"], o["out"], None,
                                               streams[i].cuda_stream)
                    else:
                        gdn.gdn_verify_lazy(dims_of(s), params_of(x), x["qkv"], x["z"], x["alpha"], x["beta_raw"], x["state"],
                                            x["conv_state"], o["out"], stream=streams[i].cuda_stream)

                def work(i):
                    torch.cuda.set_device(0)
                    start.wait()
                    try:
                        call(i, 0)
                    except gdn.GdnError as e:
                        errors.append(f"{mode} {shapes[i].name}: {e}")

                threads = [threading.Thread(target=work, args=(i,)) for i in range(len(shapes))]
                for t in threads:
                    t.start()
                for t in threads:
                    t.join()
                torch.cuda.synchronize()
                if errors:
                    print(errors, file=sys.stderr)
                    return 1
                for i in range(len(shapes)):
                    call(i, 1)
                torch.cuda.synchronize()
                if not all(torch.equal(a[1]["out"], b[1]["out"]) for a, b in zip(*sets)):
                    print("outputs differ", mode, act, d, file=sys.stderr)
                    return 1
    return 0


if __name__ == "__main__":
    sys.exit(main())
