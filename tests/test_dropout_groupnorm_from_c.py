"""include/dropout_train.h and include/groupnorm_train.h from plain C: a C99 program that includes
both, links against the library and calls what needs no GPU (launch plans, workspace sizes,
argument rejection, calls without elements).  The headers are valid C, every symbol links
without torch or C++, and a C caller sees the Python binding's values."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <stdio.h>
#include "dropout_train.h"
#include "groupnorm_train.h"

int main(void) {
  int64_t p[16];
  uint64_t step = 0;
  int i, d;
  for (d = 0; d < 2; ++d) {
    if (groupnorm_train_launch_plan(GROUPNORM_BF16, 8, 4096, 320, 32, d, p,
                                    GROUPNORM_PLAN_FIELDS) != RMSN_OK) return 1;
    printf("gn_plan%d", d);
    for (i = 0; i < GROUPNORM_PLAN_FIELDS; ++i) printf(" %lld", (long long)p[i]);
    printf("\n");
  }
  printf("gn_fwd_ws %zu\n",
         groupnorm_train_fwd_workspace_bytes(GROUPNORM_FP32, 1, 262144, 128, 32));
  printf("gn_bwd_ws %zu\n",
         groupnorm_train_bwd_workspace_bytes(GROUPNORM_FP16, 5, 1023, 640, 32));
  printf("drop_none %d\n", dropout_train_fwd(NULL, NULL, NULL, DROPOUT_BF16, 0, 0.5, 1, 0, &step,
                                             NULL));
  printf("drop_null %d\n", dropout_train_bwd(NULL, NULL, DROPOUT_FP16, 8, 0.5, 1, 0, NULL, NULL));
  printf("rms_null %d\n", rmsnorm_dropout_train_fwd(NULL, NULL, NULL, RMSN_W_BF16, NULL, NULL,
                                                    NULL, 4, 1, 64, 64, 64, 1e-6f, 0.1, 1, 0,
                                                    NULL, NULL));
  printf("rms_bwd_null %d\n", rmsnorm_dropout_train_bwd(NULL, NULL, NULL, NULL, NULL, RMSN_W_FP32,
                                                        NULL, NULL, NULL, NULL, 0, 4, 1, 64, 0.1,
                                                        1, 0, NULL, 1, NULL));
  printf("gn_null %d\n", groupnorm_train_fwd(NULL, GROUPNORM_BF16, NULL, NULL, GROUPNORM_FP32,
                                             NULL, NULL, NULL, NULL, 0, 1, 1, 64, 8, 64, 64,
                                             1e-5f, GROUPNORM_ACT_SILU, NULL));
  printf("gn_wide %d\n", groupnorm_train_bwd(NULL, NULL, GROUPNORM_BF16, NULL, NULL, NULL, NULL,
                                             GROUPNORM_FP32, NULL, NULL, NULL, NULL, 0, 1, 1,
                                             4104, 8, 4104, 4104, GROUPNORM_ACT_NONE, NULL));
  return 0;
}
"""


def test_c_program_links_and_sees_the_bindings_values(tmp_path):
    from rmsnorm_fwd_02_gb300 import _native as N
    from rmsnorm_fwd_02_gb300 import build as B
    libdir = os.path.dirname(B.build())
    src = tmp_path / "abi.c"
    src.write_text(PROGRAM)
    exe = tmp_path / "abi"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic",
                    "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe),
                    "-L", libdir, "-lrmsnorm_train", f"-Wl,-rpath,{libdir}"], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = dict(line.split(" ", 1) for line in out.strip().splitlines())
    for d in (0, 1):
        plan = N.groupnorm_train_launch_plan(N.GROUPNORM_BF16, 8, 4096, 320, 32, d)
        assert [int(v) for v in got[f"gn_plan{d}"].split()] == [
            plan[k] for k in N.GROUPNORM_PLAN_FIELDS]
    assert int(got["gn_fwd_ws"]) == N.groupnorm_train_fwd_workspace_bytes(
        N.GROUPNORM_FP32, 1, 262144, 128, 32) > 0
    assert int(got["gn_bwd_ws"]) == N.groupnorm_train_bwd_workspace_bytes(
        N.GROUPNORM_FP16, 5, 1023, 640, 32) > 0
    want = {"drop_none": 0, "drop_null": 1, "rms_null": 1, "rms_bwd_null": 1, "gn_null": 1,
            "gn_wide": 2}  # RMSN_OK, _ERR_INVALID_ARG, _ERR_UNSUPPORTED
    assert {k: int(got[k]) for k in want} == want
