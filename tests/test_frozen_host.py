"""Host code of the operators on frozen 4-bit weights that needs no GPU: small programs compiled against the library's
own headers, and refusals in front of any launch."""
import os
import subprocess
import textwrap

import pytest
import torch

import weight_only_int4_wise_b200 as w
from weight_only_int4_wise_b200 import build


def compile_and_run(tmp_path, name, source, flags=()):
    """Compiles a C++ program that includes headers of csrc/ and returns its completed run."""
    cpp, exe = os.path.join(tmp_path, name + ".cpp"), os.path.join(tmp_path, name)
    with open(cpp, "w") as out:
        out.write(textwrap.dedent(source))
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", build.CSRC, *flags, cpp, "-o", exe, "-pthread"],
                   check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=120)


def test_every_warp_indexes_inside_the_parameter_arrays(tmp_path):
    # The set-up of the transposed and wide gated products runs on all warps, the producer's and the MMA issuer's too:
    # the block that indexes the arrays of two weight matrices is 0 or 1 for each, and the groups share out all stages.
    run = compile_and_run(tmp_path, "roles", """
        #include <cstdio>
        #include "roles.h"
        int main() {
            const int forms[][2] = {{1, 2}, {1, 4}, {2, 4}};  // blocks per CTA, decoding groups
            for (auto& form : forms) {
                const int km = form[0], groups = form[1], turn = groups / km;
                int taken[2][4] = {};
                for (int warp = 0; warp < w4a16::kFirstDecodeWarp + w4a16::kGroupWarps * groups; ++warp) {
                    const int block = w4a16::block_of_warp(warp, km), stage = w4a16::stage_of_warp(warp, km);
                    if (block < 0 || block >= km || stage < 0 || stage >= turn) {
                        std::printf("warp %d of (%d, %d): block %d, stage %d\\n", warp, km, groups, block, stage);
                        return 1;
                    }
                    if (warp >= w4a16::kFirstDecodeWarp) ++taken[block][stage];
                }
                for (int b = 0; b < km; ++b)
                    for (int s = 0; s < turn; ++s)
                        if (taken[b][s] != w4a16::kGroupWarps) return 2;
            }
            return 0;
        }
    """)
    assert run.returncode == 0, run.stdout


def test_threads_that_make_first_calls_at_once_do_not_race(tmp_path):
    # Under the race detector: eight threads prepare two devices at once; each device is prepared once, a failure is
    # tried again, and what the preparation wrote is there for every thread that finds it done.
    run = compile_and_run(tmp_path, "once", """
        #include <cstdio>
        #include <thread>
        #include <vector>
        #include "once.h"
        static w4a16::OncePerDevice once;
        static int tries[2], prepared[2];  // plain: the class has to order them
        int main() {
            std::vector<std::thread> threads;
            std::atomic<int> wrong{0};
            for (int t = 0; t < 8; ++t)
                threads.emplace_back([t, &wrong] {
                    const int dev = t & 1;
                    for (int i = 0; i < 1000; ++i) {
                        const int rc = once.run(dev, [dev] {
                            if (++tries[dev] == 1) return 3;
                            prepared[dev] += 1;
                            return 0;
                        });
                        if (rc == 0 && prepared[dev] != 1) wrong.fetch_add(1);
                        if (rc != 0 && rc != 3) wrong.fetch_add(1);
                    }
                });
            for (auto& t : threads) t.join();
            return wrong.load() || tries[0] != 2 || tries[1] != 2;
        }
    """, flags=("-fsanitize=thread",))
    if "unexpected memory mapping" in run.stderr:
        pytest.skip("the race detector does not start under this kernel's address layout")
    assert run.returncode == 0, run.stdout + run.stderr


def test_no_launch_keeps_an_unguarded_table():
    for path in build.sources():
        with open(path) as source:
            assert "attr_done" not in source.read(), path


def test_outputs_that_would_not_be_written_are_refused():
    rows, wt, S = torch.zeros((4, 64)).half(), torch.zeros(4096, dtype=torch.uint8), torch.ones((1, 64)).half()
    out = torch.zeros((4, 64)).half()
    for names in (("out_gate",), ("out_up",), ("out_gate", "out_up")):
        with pytest.raises(ValueError, match="save=True"):
            w.gated_gemm(rows, wt, S, wt, S, 64, 64, **{n: out for n in names})
